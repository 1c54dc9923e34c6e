"""GPU parity of the scored router, its gradient and its bias step with the fp64 oracle.

Ids and device masks are equal.  With u = 2^-24 (half a unit of fp32): an exponential
is within 4 u and its argument's rounding |argument| u, 1 + e and a division add 2 u, a
softmax's sum of 256 terms at most 16 u: a score is within S = (24 + 2 |z|max) u of
itself.  Renormalising adds a sum of 16 (5 u), a division and the scale: a gate is within
2 S + 8 u.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import scored

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SENTINEL = -77


@pytest.fixture(scope="module")
def occ():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_top_route_gb300 import build
    build.build()
    import combine_top_route_gb300 as occ
    occ.lib()
    return occ


def logits_of(T, Ne, seed=0, rounded=False):
    rng = np.random.default_rng(seed)
    boost = rng.random((8, Ne)) < 0.2
    z = (rng.normal(size=(T, Ne)) + 2.0 * boost[rng.integers(0, 8, T)] - 1).astype(np.float32)
    if rounded:   # many equal logits
        z = np.round(z * 4) / 4
    return z


def place(Ne, Nd, seed=0):
    return np.random.default_rng(seed + 99).permutation(np.arange(Ne) % Nd).astype(np.int32)


def setup(occ, z, k, Nd, renorm=True, sigmoid=True, n_groups=1, keep=1, best=1, by_vdev=False,
          scale=1.0, bias_rate=0.0):
    T, Ne = z.shape
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, n_experts=Ne, top_k=k, n_vdev=Nd,
                                                       renorm=renorm))
    opt = occ.occult_score_t(score=occ.SCORE_SIGMOID if sigmoid else occ.SCORE_SOFTMAX,
                             n_groups=n_groups, keep_groups=keep, group_best=best,
                             group_kind=occ.GROUP_VDEV if by_vdev else occ.GROUP_BLOCKS,
                             scale=scale, bias_rate=bias_rate)
    return ds, opt


def gpu(a, dt=torch.float32):
    return None if a is None else torch.as_tensor(np.ascontiguousarray(a)).to(dt).cuda()


def run(occ, z, k, e2v, Nd, bias=None, stream=None, **kw):
    T, Ne = z.shape
    ds, opt = setup(occ, z, k, Nd, **kw)
    new = lambda n, dt: torch.full((n + 8,), SENTINEL, dtype=dt, device="cuda")  # noqa: E731
    ids, gates, vm = new(T * k, torch.int32), new(T * k, torch.float32), new(T, torch.int32)
    occ.occult_route_scored(ds, opt, gpu(z), gpu(e2v, torch.int32), ids, gates, vm, bias=gpu(bias),
                            stream=stream)
    torch.cuda.synchronize()
    assert (ids[T * k:] == SENTINEL).all() and (gates[T * k:] == SENTINEL).all()
    assert (vm[T:] == SENTINEL).all()
    return (ids[:T * k].view(T, k).cpu().numpy(), gates[:T * k].view(T, k).double().cpu().numpy(),
            vm[:T].cpu().numpy().astype(np.int64) & 0xffffffff)


def score_err(z):
    fin = z[np.isfinite(z) & (z > scored.LOWEST)]
    return (24 + 2 * (np.abs(fin).max() if fin.size else 0)) * U


def check(occ, z, k, Nd, bias=None, seed=0, **kw):
    e2v = place(z.shape[1], Nd, seed)
    ids, gates, vm = run(occ, z, k, e2v, Nd, bias, **kw)
    want = scored.route(z, k, e2v, bias=bias, **kw)
    assert (ids == want[0]).all(), np.argwhere(ids != want[0])[:4]
    assert (vm == want[2]).all()
    err = (2 * score_err(z) + 8 * U) * np.abs(want[1]) + 1e-37
    assert (np.abs(gates - want[1]) <= err).all(), np.max(np.abs(gates - want[1]) - err)
    return ids


SIZES = [(1, 64, 8, 8), (7, 8, 2, 4), (257, 60, 4, 4), (300, 33, 3, 1), (129, 96, 12, 32),
         (513, 128, 16, 16), (333, 256, 8, 32), (64, 1, 1, 1), (50, 2, 2, 2), (90, 255, 5, 5),
         (31, 16, 16, 4), (1000, 64, 8, 8)]


@pytest.mark.parametrize("T,Ne,k,Nd", SIZES)
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("biased", [True, False])
def test_sizes(occ, T, Ne, k, Nd, sigmoid, biased):
    bias = np.random.default_rng(T).normal(size=Ne).astype(np.float32) * 0.1 if biased else None
    check(occ, logits_of(T, Ne, T), k, Nd, bias, sigmoid=sigmoid, renorm=biased, scale=2.5)


@pytest.mark.parametrize("Ne,G,keep,k", [(64, 8, 4, 8), (256, 8, 4, 8), (60, 3, 1, 4), (60, 2, 2, 16),
                                         (96, 32, 5, 12), (32, 32, 16, 16), (8, 4, 1, 2),
                                         (160, 5, 3, 6), (256, 2, 1, 16), (33, 11, 4, 3)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_groups(occ, Ne, G, keep, k, best, sigmoid):
    rng = np.random.default_rng(Ne)
    for by_vdev in (False, True):
        for bias in (None, (rng.normal(size=Ne) * 0.2).astype(np.float32)):
            check(occ, logits_of(200, Ne, G), k, G if by_vdev or Ne % 4 else 4, bias,
                  sigmoid=sigmoid, n_groups=G, keep=keep, best=best, by_vdev=by_vdev)


@pytest.mark.parametrize("Ne,G,keep", [(64, 1, 1), (64, 8, 2), (60, 4, 2), (256, 8, 3)])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_switched_off(occ, Ne, G, keep, biased, sigmoid):
    """-inf and the lowest value, groups and rows without an expert left, fewer than k."""
    rng = np.random.default_rng(5)
    z = logits_of(120, Ne, 3)
    z[rng.random(z.shape) < 0.5] = -np.inf
    z[rng.random(z.shape) < 0.2] = scored.LOWEST
    z[3] = -np.inf
    z[4] = scored.LOWEST
    z[5, 2:] = -np.inf
    z[6, :Ne // 2] = -np.inf
    z[7, :-1] = -np.inf
    bias = (rng.normal(size=Ne) * 2).astype(np.float32) if biased else None
    check(occ, z, 6, 4, bias, n_groups=G, keep=keep, best=2, sigmoid=sigmoid)


@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_ties(occ, biased, sigmoid):
    """Equal logits, equal rows, an all-zero router: the lower expert, the lower group."""
    z = logits_of(150, 64, 8, rounded=True)
    z[0] = 0
    z[1] = 1.5
    z[2, ::2] = 0.25
    bias = np.zeros(64, np.float32) if biased else None
    check(occ, z, 8, 8, bias, sigmoid=sigmoid)
    check(occ, z, 8, 8, bias, sigmoid=sigmoid, n_groups=8, keep=3, best=2)


def test_near_ties_fall_as_in_64_bits(occ):
    """Ranks closer than fp32 can tell apart, within the list, at its end and between
    groups: biases that even out the scores of neighbours to a few 1e-9."""
    rng = np.random.default_rng(12)
    Ne, T = 64, 400
    z = rng.normal(size=(T, Ne)).astype(np.float32)
    z[:] = z[0]                         # one row: its biases make all ranks nearly equal
    s = scored.scores(z[0], True)[0]
    bias = (1.0 - s).astype(np.float32)   # ranks 1 +- 2^-25: rounding decides
    z[1:] += (rng.integers(-2, 3, size=(T - 1, Ne)) * 2.0 ** -22).astype(np.float32)
    check(occ, z, 8, 8, bias)
    check(occ, z, 8, 8, bias, n_groups=8, keep=4, best=2)
    # far tails: scores far below the rank's rounding
    z = (rng.normal(size=(100, Ne)) * 30).astype(np.float32)
    for sigmoid in (True, False):
        check(occ, z, 6, 8, (0.25 * rng.integers(0, 3, Ne)).astype(np.float32), sigmoid=sigmoid)
        check(occ, z, 6, 8, None, sigmoid=sigmoid, n_groups=4, keep=2, best=2)


def test_nan_and_infinity_leave_valid_ids(occ):
    """Whatever a row holds, its ids are k different experts and the neighbours' rows as usual."""
    rng = np.random.default_rng(1)
    z = logits_of(64, 32, 2)
    z[::3][rng.random(z[::3].shape) < 0.3] = np.nan
    z[9] = np.nan
    z[12] = np.inf
    z[15, 4] = np.inf
    for bias in (None, np.where(np.arange(32) % 7 == 0, np.nan, 0.1).astype(np.float32),
                 np.where(np.arange(32) % 5 == 0, -np.inf, 0.1).astype(np.float32)):
        for sigmoid in (True, False):
            e2v = place(32, 4)
            ids, _, _ = run(occ, z, 5, e2v, 4, bias, sigmoid=sigmoid, n_groups=4, keep=2, best=2)
            assert ((ids >= 0) & (ids < 32)).all()
            assert all(len(set(r)) == 5 for r in ids.tolist())
    ids = check(occ, np.where(np.isnan(z) | np.isinf(z), -np.inf, z), 5, 4)
    got = run(occ, np.where(np.isinf(z), -np.inf, z), 5, place(32, 4), 4)   # NaN ranks as switched off
    assert (got[0] == ids).all()


def test_grad(occ):
    rng = np.random.default_rng(3)
    for T, Ne, k, Nd in SIZES:
        for sigmoid in (True, False):
            for renorm in (True, False):
                z = logits_of(T, Ne, T + 1)
                if Ne > 4:
                    z[rng.random(z.shape) < 0.2] = -np.inf
                    z[0] = -np.inf
                e2v = place(Ne, Nd)
                kw = dict(sigmoid=sigmoid, scale=1.7, renorm=renorm)
                ids = scored.route(z, k, e2v, **kw)[0].astype(np.int32)
                if T > 40:
                    ids[5, 0] = -1       # a dropped slot
                dg = rng.normal(size=(T, k)).astype(np.float32)
                ds, opt = setup(occ, z, k, Nd, **kw)
                out = torch.full((T * Ne + 8,), float(SENTINEL), device="cuda")
                occ.occult_route_scored_grad(ds, opt, gpu(z), gpu(ids, torch.int32), gpu(dg), out)
                torch.cuda.synchronize()
                assert (out[T * Ne:] == SENTINEL).all()
                got = out[:T * Ne].view(T, Ne).double().cpu().numpy()
                want = scored.grad(z, ids, dg, **kw)
                # magnitudes that cancel: every ds_j is of size |u|max / S (renormalised), and
                # each of at most four factors is within 2 S + 24 u of itself, 1 - s within
                # 8 u of the size of 1
                s = np.array([scored.scores(r, sigmoid)[0] for r in z])
                S = np.array([max(1e-30, s[t][[e for e in ids[t] if e >= 0]].sum()) for t in range(T)])
                big = 1.7 * np.abs(dg).max(axis=1) * (2 / S if renorm else 1)
                err = (6 * score_err(z) + 60 * U) * big[:, None] * s * (1 if sigmoid else 2) + 1e-36
                assert (np.abs(got - want) <= err).all(), (T, Ne, sigmoid, renorm)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("low", [0.0, -85.0])
def test_an_only_expert_has_the_whole_gate(occ, sigmoid, low):
    """One expert a token, renormalised: its gate is the scale (to the fast division's two units,
    2^-22) and has no gradient, exactly (s / s is 1 in IEEE arithmetic), however small its
    score."""
    T, Ne = 257, 62
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, n_experts=Ne, top_k=1, n_vdev=2, renorm=1))
    opt = occ.occult_score_t(occ.SCORE_SIGMOID if sigmoid else occ.SCORE_SOFTMAX, scale=2.5)
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = low + torch.randn(T, Ne, generator=g, device="cuda")
    ids, vmask = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
    gates, dgates = torch.empty(T, device="cuda"), torch.randn(T, generator=g, device="cuda")
    dlogits = torch.full((T, Ne), 7.0, device="cuda")
    e2v = (torch.arange(Ne, device="cuda") % 2).int()
    occ.occult_route_scored(ds, opt, logits, e2v, ids, gates, vmask)
    occ.occult_route_scored_grad(ds, opt, logits, ids, dgates, dlogits)
    assert (ids.long() == logits.argmax(1)).all()
    assert (gates.double() / 2.5 - 1).abs().max() <= 2.0 ** -22 and (dlogits == 0).all()


def test_grad_is_the_difference_quotient(occ):
    """The kernel's own gates, moved along random directions, against its gradient."""
    rng = np.random.default_rng(7)
    T, Ne, k = 16, 32, 4
    z = logits_of(T, Ne, 21).astype(np.float32)
    e2v, dg = place(Ne, 4), rng.normal(size=(T, k)).astype(np.float32)
    for kw in (dict(sigmoid=True, renorm=True), dict(sigmoid=True, renorm=False),
               dict(sigmoid=False, renorm=True), dict(sigmoid=False, renorm=False)):
        ids = run(occ, z, k, e2v, 4, **kw)[0]
        ds, opt = setup(occ, z, k, 4, **kw)
        out = torch.empty(T * Ne, device="cuda")
        occ.occult_route_scored_grad(ds, opt, gpu(z), gpu(ids, torch.int32), gpu(dg), out)
        way = rng.normal(size=z.shape).astype(np.float32)
        h = 2.0 ** -9
        up, lo = ((z + sgn * h * way).astype(np.float32) for sgn in (1, -1))
        fix = lambda zz: np.stack([  # noqa: E731  (the gates of the same choice)
            (lambda s: s / s.sum() if kw["renorm"] else s)(scored.scores(zz[t], kw["sigmoid"])[0][ids[t]])
            for t in range(T)])
        num = (dg * (fix(up) - fix(lo))).sum() / (2 * h)
        ana = (out.view(T, Ne).double().cpu().numpy() * way).sum()
        # third derivatives are below 1 a term of T k: h^2 / 6 of that, and fp32's roundings
        # of the points, 2^-22 / h a term
        assert abs(num - ana) < T * k * (h * h * np.abs(way).max() ** 3 + 2.0 ** -22 / h)


def test_bias_step(occ):
    rng = np.random.default_rng(2)
    for G, Ne in ((1, 64), (5, 256), (3, 1)):
        counts = rng.integers(0, 9, size=(G, Ne)).astype(np.int32)
        bias = rng.normal(size=Ne).astype(np.float32)
        ds, opt = setup(occ, np.zeros((4, Ne), np.float32), 1, 1, bias_rate=1e-3)
        b = gpu(bias)
        occ.occult_route_bias_step(ds, opt, gpu(counts, torch.int32), b)
        want = bias + np.float32(1e-3) * np.sign(scored.bias_step(np.zeros(Ne), counts, 1.0)).astype(np.float32)
        assert (b.cpu().numpy() == want.astype(np.float32)).all()


def test_streams_graphs_and_odd_addresses(occ):
    """Another stream, a replayed graph on new logits, buffers off a 16-byte boundary, no tokens."""
    T, Ne, k = 100, 60, 4
    e2v = place(Ne, 4)
    za, zb = logits_of(T, Ne, 1), logits_of(T, Ne, 2)
    want = [scored.route(z, k, e2v, n_groups=4, keep=2, best=2) for z in (za, zb)]
    ds, opt = setup(occ, za, k, 4, n_groups=4, keep=2, best=2)
    odd = lambda n, dt=torch.float32: torch.zeros(n + 1, dtype=dt, device="cuda")[1:]  # noqa: E731
    z, ids, gates, vm = odd(T * Ne), odd(T * k, torch.int32), odd(T * k), odd(T, torch.int32)
    dz, dg = odd(T * Ne), gpu(np.ones((T, k)))
    ev = odd(Ne, torch.int32)
    ev.copy_(gpu(e2v, torch.int32))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def both(stream):
        occ.occult_route_scored(ds, opt, z, ev, ids, gates, vm, stream=stream)
        occ.occult_route_scored_grad(ds, opt, z, ids, dg, dz, stream=stream)

    z.copy_(gpu(za).view(-1))
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    s.synchronize()
    assert (ids.view(T, k).cpu().numpy() == want[0][0]).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(None)
    for zz, w in ((zb, want[1]), (za, want[0])):
        z.copy_(gpu(zz).view(-1))
        g.replay()
        torch.cuda.synchronize()
        assert (ids.view(T, k).cpu().numpy() == w[0]).all()
        ref = scored.grad(zz, w[0], np.ones((T, k)))
        assert np.abs(dz.view(T, Ne).cpu().numpy() - ref).max() < 1e-4
    empty = ds.replace(T=0)
    occ.occult_route_scored(empty, opt, z[:0], ev, ids[:0], gates[:0], vm[:0])
    occ.occult_route_scored_grad(empty, opt, z[:0], ids[:0], dg[:0], dz[:0])


def test_the_layer_takes_the_routing(occ):
    """ids, gates and masks feed the BRIM build: every kept slot gets one EPD row."""
    T, Ne, k, Nd = 300, 64, 8, 8
    z = logits_of(T, Ne, 6)
    placement = np.random.default_rng(1).permutation(Ne).reshape(Nd, -1).astype(np.int32)
    e2v = np.empty(Ne, np.int32)
    for d in range(Nd):
        e2v[placement[d]] = d
    ds, opt = setup(occ, z, k, Nd, n_groups=8, keep=3, best=2, by_vdev=True)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, gates, vm = i32(T, k), torch.zeros(T, k, device="cuda"), i32(T)
    occ.occult_route_scored(ds, opt, gpu(z), gpu(e2v, torch.int32), ids, gates, vm)
    counts, exp_off = i32(4), i32(Ne + 1)
    ws = torch.zeros(occ.workspace_size(ds, occ.WS_BUILD_BRIM), dtype=torch.uint8, device="cuda")
    occ.occult_build_brim(ds, ids, gates, vm, gpu(placement, torch.int32), i32(Nd, T), i32(Nd + 1),
                          i32(Ne, T), exp_off, i32(T * k), torch.zeros(T * k, device="cuda"), counts, ws)
    c = counts.cpu().tolist()
    assert c[1] == T * k and c[2] <= 3
    per = np.bincount(ids.cpu().numpy().ravel(), minlength=Ne)[placement.ravel()]
    assert (np.diff(exp_off.cpu().numpy()) == per).all()


@pytest.mark.parametrize("sigmoid", [True, False])
def test_more_tokens_than_warps(occ, sigmoid):
    z = logits_of(20011, 32, 1)
    bias = (np.random.default_rng(3).normal(size=32) * 0.1).astype(np.float32)
    check(occ, z, 4, 4, bias, sigmoid=sigmoid, n_groups=4, keep=2, best=2)
    e2v, kw = place(32, 4), dict(sigmoid=sigmoid, scale=1.0, renorm=True)
    ids = scored.route(z, 4, e2v, **kw)[0].astype(np.int32)
    dg = np.random.default_rng(5).normal(size=(20011, 4)).astype(np.float32)
    ds, opt = setup(occ, z, 4, 4, **kw)
    out = torch.full((20011 * 32,), float(SENTINEL), device="cuda")
    occ.occult_route_scored_grad(ds, opt, gpu(z), gpu(ids, torch.int32), gpu(dg), out)
    want = scored.grad(z, ids, dg, **kw)
    got = out.view(20011, 32).double().cpu().numpy()
    # (see test_grad: at most twice the largest |dgate| over a sum of four scores)
    s = np.array([scored.scores(r, sigmoid)[0] for r in z])
    S = np.take_along_axis(s, ids.astype(np.int64), 1).sum(axis=1)
    err = (6 * score_err(z) + 60 * U) * (2 * np.abs(dg).max(axis=1) / S)[:, None] * s * 2 + 1e-36
    assert (np.abs(got - want) <= err).all()


def grad_of(occ, z, ids, dg, **kw):
    """The kernel's dlogits for a given choice."""
    (T, Ne), k = z.shape, ids.shape[1]
    ds, opt = setup(occ, z, k, 1, **kw)
    out = torch.full((T * Ne + 8,), float(SENTINEL), device="cuda")
    occ.occult_route_scored_grad(ds, opt, gpu(z), gpu(ids, torch.int32), gpu(dg), out)
    torch.cuda.synchronize()
    assert (out[T * Ne:] == SENTINEL).all()
    return out[:T * Ne].view(T, Ne).double().cpu().numpy()


def chosen(rng, T, Ne, k):
    return np.stack([rng.permutation(Ne)[:k] for _ in range(T)]).astype(np.int32)


@pytest.mark.parametrize("sigmoid", [True, False])
def test_grad_of_scores_near_the_end_of_the_range(occ, sigmoid):
    """Chosen scores whose sum is below fp32's normal numbers: shares of it, and no infinity.

    A score is then within a unit of the subnormals, 2^-149, besides its relative error; a
    sigmoid below 2^-128 is 0 (its exponential is infinite).  With e_j the errors of the
    scores, a share s_j / S moves by (e_j + share sum e) / S, the mean of the u_i by |u|max
    times the sum of those.
    """
    rng = np.random.default_rng(11)
    T, Ne, k = 80, 16, 4
    z = rng.uniform(-88.6, -87.0, size=(T, Ne)).astype(np.float32)
    ids = chosen(rng, T, Ne, k)
    if sigmoid:
        z[::5, ::2] = -100.0          # of scores that are 0 beside these
        z[1] = -100.0
        z[2, ids[2, :2]] = -88.3, -88.5
        ids[2, 2:] = -1
        known = np.where(z < -88.73, -np.inf, z)
    else:
        z[:, 0] = 0.0                 # an expert that the bias keeps out has nearly everything
        ids = 1 + chosen(rng, T, Ne - 1, k)
        known = z
    dg = rng.choice([3.0, -3.0, 0.5], size=(T, k)).astype(np.float32)
    got = grad_of(occ, z, ids, dg, sigmoid=sigmoid, renorm=True, scale=2.5)
    assert np.isfinite(got).all()
    want = scored.grad(known, ids, dg, sigmoid=sigmoid, renorm=True, scale=2.5)
    s = np.array([scored.scores(r, sigmoid)[0] for r in known])
    for t in range(T):
        live = [e for e in ids[t] if e >= 0]
        S, big = max(s[t, live].sum(), 2.0 ** -149), 2.5 * 2 * np.abs(dg[t]).max()
        e = score_err(known) * s[t] + 2.0 ** -149
        err = np.full(Ne, 1e-12)      # (the oracle's own sum of ds s, which is 0, over scores up to 1)
        err[live] += big * (e[live] + s[t, live] / S * 3 * e[live].sum()) / S + 60 * U * big * s[t, live] / S
        assert (np.abs(got[t] - want[t]) <= err).all(), (t, np.max(np.abs(got[t] - want[t]) / err))


def grad_bound(z, ids, dg, sigmoid, renorm, scale, rel):
    """Errors of dlogits relative to what each is the sum of.

    With c = 1 - s of sigmoids and p_j = s_j / S, renormalised: dz_j = p_j c_j (u_j - sum p_i u_i)
    = p_j c_j sum p_i (u_j - u_i): `rel` of p_j c_j sum p_i |u_j - u_i|, and k + 2 times that, since
    the differences are taken from the largest share's u (p >= 1 / k) first.  Otherwise, sigmoid:
    `rel` of itself; softmax: `rel` of s_e (|v_e| (1 - s_e) + sum over the others of |v_i| s_i),
    v the u of an expert, 0 where it is not chosen.
    """
    T, Ne = z.shape
    err = np.zeros((T, Ne))
    for t in range(T):
        s = scored.scores(z[t], sigmoid)[0]
        live = [(scale * float(u), e) for u, e in zip(dg[t], ids[t]) if e >= 0]
        c = {e: 1 / (1 + np.exp(float(z[t, e]))) if sigmoid else 1.0 for _, e in live}
        if renorm:
            S = sum(s[e] for _, e in live)
            for u, e in live:
                err[t, e] = rel * (len(live) + 2) * s[e] / S * c[e] * sum(s[i] / S * abs(u - v) for v, i in live)
        elif sigmoid:
            for u, e in live:
                err[t, e] = rel * abs(u) * s[e] * c[e]
        else:
            v = np.zeros(Ne)
            for u, e in live:
                v[e] += u
            rest = np.array([s[np.arange(Ne) != e].sum() for e in range(Ne)])   # 1 - s, without the cancellation
            rest_v = np.array([(np.abs(v) * s)[np.arange(Ne) != e].sum() for e in range(Ne)])
            err[t] = rel * s * (np.abs(v) * rest + rest_v)
    return err


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_grad_where_one_expert_has_nearly_all(occ, sigmoid, renorm):
    """A share, or a softmax's score, within 1e-3 to 1e-11 of 1: its gradient is as small as the
    others' together, and keeps its digits."""
    rng = np.random.default_rng(17)
    T, Ne, k = 96, 60, 5
    z = rng.normal(size=(T, Ne)).astype(np.float32) - 24
    ids, dg = chosen(rng, T, Ne, k), rng.normal(size=(T, k)).astype(np.float32)
    lead = rng.uniform(-14, 2, size=T).astype(np.float32)      # 10 to 26 above the others
    z[np.arange(T), ids[np.arange(T), np.arange(T) % k]] = lead
    ids[5] = chosen(rng, 1, Ne, k)      # one that is not chosen may have it
    kw = dict(sigmoid=sigmoid, renorm=renorm, scale=1.7)
    got = grad_of(occ, z, ids, dg, **kw)
    want = np.zeros_like(got)
    for t in range(T):
        s, u = scored.scores(z[t], sigmoid)[0], 1.7 * dg[t].astype(np.float64)
        c = 1 / (1 + np.exp(z[t].astype(np.float64))) if sigmoid else np.ones(Ne)
        p = s[ids[t]] / s[ids[t]].sum()
        if renorm:
            want[t, ids[t]] = p * c[ids[t]] * (p * (u[:, None] - u)).sum(axis=1)
        elif sigmoid:
            want[t, ids[t]] = u * s[ids[t]] * c[ids[t]]
        else:
            v = np.zeros(Ne)
            v[ids[t]] = u
            want[t] = [s[e] * (s * (v[e] - v)).sum() for e in range(Ne)]
    # (a sum of 60 exponentials besides: 8 u)
    rel = 6 * score_err(z) + 80 * U
    off, err = np.abs(got - want), grad_bound(z, ids, dg, rel=rel, **kw) + 1e-37
    assert (off <= err).all(), np.max(off / err)


@pytest.mark.parametrize("renorm", [True, False])
def test_grad_of_sure_sigmoids(occ, renorm):
    """Logits of 8 to 40: 1 - s keeps its digits (the exponential's 4 u, two sums and divisions of
    u each, s and the products: 24 u; renormalised the shares' errors besides)."""
    rng = np.random.default_rng(13)
    T, Ne, k = 120, 32, 4
    z = rng.uniform(8, 40, size=(T, Ne)).astype(np.float32)
    z[::3] = rng.uniform(-4, 10, size=z[::3].shape)
    z[1::3, ::2] -= 40
    ids, dg = chosen(rng, T, Ne, k), rng.normal(size=(T, k)).astype(np.float32)
    kw = dict(sigmoid=True, renorm=renorm, scale=1.7)
    got = grad_of(occ, z, ids, dg, **kw)
    # (the formula with 1 - s as 1 / (1 + e^z))
    want = np.zeros_like(got)
    for t in range(T):
        s = scored.scores(z[t], True)[0][ids[t]]
        u = 1.7 * dg[t].astype(np.float64)
        c = 1 / (1 + np.exp(z[t, ids[t]].astype(np.float64)))
        p = s / s.sum()
        want[t, ids[t]] = p * c * (p * (u[:, None] - u)).sum(axis=1) if renorm else u * s * c
    rel = 6 * score_err(z) + 60 * U if renorm else 24 * U
    assert (np.abs(got - want) <= grad_bound(z, ids, dg, rel=rel, **kw) + 1e-37).all()


@pytest.mark.parametrize("Ne,G,keep,k", [(64, 8, 4, 6), (48, 3, 2, 4), (256, 8, 4, 8), (60, 4, 1, 4)])
@pytest.mark.parametrize("best", [1, 2])
def test_groups_of_small_worth(occ, Ne, G, keep, k, best):
    """Groups whose scores all lie far below the largest, or far below 1: still by their worth."""
    rng = np.random.default_rng(Ne + best)
    for spread in (10.0, 30.0):
        z = (rng.normal(size=(150, Ne)) * spread).astype(np.float32)
        for sigmoid in (False, True):
            for by_vdev in (False, True):
                check(occ, z, k, G if by_vdev else 4, None, sigmoid=sigmoid, n_groups=G, keep=keep, best=best,
                      by_vdev=by_vdev)
    for low in (-45.0, -80.0):
        z = (low + rng.normal(size=(150, Ne))).astype(np.float32)
        check(occ, z, k, 4, None, n_groups=G, keep=keep, best=best)
        check(occ, z, k, 4, None, sigmoid=False, n_groups=G, keep=keep, best=best)
    # one group of eight equal logits, and two whose best are a factor e apart, 33 below
    z = np.full((4, 48), -60.0, np.float32)
    z[:, :8], z[:, 20], z[:, 40] = 0.0, -34.0, -33.0
    z[1, [21, 41]] = -34.0, -33.0
    z[2, [20, 40]], z[3, [20, 40]] = (-33.0, -34.0), (-34.0, -34.0)
    for sigmoid in (False, True):
        ids = check(occ, z, 9, 4, None, sigmoid=sigmoid, n_groups=3, keep=2, best=best, renorm=False)
        assert ids[:, 8].tolist() == [40, 40, 20, 20]


@pytest.mark.parametrize("biased", [True, False])
def test_groups_of_equal_worth(occ, biased):
    """sigmoid(x) + sigmoid(-x) is 1 for every x: such groups are equal, and the lower one is kept,
    whatever the bias of the pair adds up to; a hair more and the higher one is."""
    rng = np.random.default_rng(19)
    T, G, per = 200, 8, 4
    x = rng.uniform(0, 12, size=(T, G)).astype(np.float32)
    z = np.full((T, G, per), -np.inf, np.float32)
    z[:, :, 1], z[:, :, 3] = x, -x
    bias = np.zeros((G, per), np.float32)
    if biased:     # halves and quarters that cancel in every pair, whichever stands first
        b = rng.integers(-3, 4, size=G).astype(np.float32) / 4
        bias[:, 1], bias[:, 3] = 3 + b, 3 - b
    kw = dict(n_groups=G, keep=3, best=2, renorm=False)
    z, bias = z.reshape(T, -1), bias.reshape(-1) if biased else None
    ids = check(occ, z, 6, 4, bias, **kw)
    assert (np.sort(ids, axis=1) == [1, 3, 5, 7, 9, 11]).all()
    up = z.copy()
    up[:, 7 * per + 3] += np.maximum(np.abs(up[:, 7 * per + 3]), 1) * np.float32(2.0 ** -20)
    ids = check(occ, up, 6, 4, bias, **kw)
    assert (np.sort(ids, axis=1) == [1, 3, 5, 7, 29, 31]).all()


@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("G,keep,best", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_nan_logits_rank_as_switched_off(occ, biased, sigmoid, G, keep, best):
    """A NaN logit leaves the choice among its row's other experts as if it were -inf; a
    softmax's gates of that row are NaN, as the formula's are, a sigmoid's others what they are."""
    rng = np.random.default_rng(23)
    z = logits_of(90, 64, 9)
    nan = rng.random(z.shape) < 0.1
    nan[::3] = False
    nan[1, 1:] = True
    bias = (rng.normal(size=64) * 0.05).astype(np.float32) if biased else None
    kw = dict(sigmoid=sigmoid, n_groups=G, keep=keep, best=best, renorm=False)
    want = check(occ, np.where(nan, np.float32(-np.inf), z), 6, 4, bias, **kw)
    ids, gates, _ = run(occ, np.where(nan, np.float32(np.nan), z), 6, place(64, 4), 4, bias, **kw)
    assert (ids == want).all()
    bad = np.take_along_axis(nan, want, 1)      # (chosen where nothing else is left)
    if sigmoid:
        assert (np.isnan(gates) == bad).all()
    else:
        assert (np.isnan(gates) == nan.any(axis=1)[:, None]).all()


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_grad_of_one_expert_in_two_slots(occ, sigmoid, renorm):
    """Slots of one expert, which the router does not write, add up: where they are its row's
    leading one as well, and beside a dropped slot."""
    rng = np.random.default_rng(29)
    T, Ne, k = 60, 40, 5
    z = logits_of(T, Ne, 4)
    ids, dg = chosen(rng, T, Ne, k), rng.normal(size=(T, k)).astype(np.float32)
    ids[:, 3] = ids[:, 1]
    ids[::4, 4] = -1
    z[np.arange(0, T, 2), ids[::2, 1]] += 9
    kw = dict(sigmoid=sigmoid, renorm=renorm, scale=1.7)
    got, want = grad_of(occ, z, ids, dg, **kw), scored.grad(z, ids, dg, **kw)
    # (a sum of 40 exponentials besides; the oracle's own differences, 2^-50 of the size of the terms)
    err = 2 * grad_bound(z, ids, dg, rel=6 * score_err(z) + 80 * U, **kw) + 2.0 ** -50 * 2 * np.abs(dg).max()
    assert (np.abs(got - want) <= err).all(), np.max(np.abs(got - want) / err)
