"""GPU parity of the output head (occult_head_loss, occult_head_step) with the fp64 oracle.

Tolerances, with u = 2^-24.  A logit: its products are exact in fp32, each 16-deep step
of the tensor cores (each product of the fp32 units) adds one rounding of at most 2 u of
a = sum |x_i w_i|: ez = (d / 16 + 8) 2 u a (fp32: (d + 8) 2 u a).  A row's log-sum: ez, the exponentials
(2^-22) and their arguments' rounding, 128 additions one after the other and their
joining, 300 u in all, and 4 u of itself.  A probability: that twice, and in training
steps of bf16 layers the kept logits' half step, s ln 2 / 2 with s = max(24, 20 tau) /
65535 octaves (over tau for the tempered one), and what lies under their range, 2^-20 of
the row's largest.  The gradient of a logit is rounded once to bf16 (2^-8), the sums of
dx and dw add (V / 16 + 8) or (T / 16 + 8) steps of 2 u of the sum of magnitudes, the
outputs their own rounding (2^-8 or u).
"""
import numpy as np
import pytest
import torch

import synth
from oracle import head as ohead

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SENTINEL = -77.0


@pytest.fixture(scope="module")
def occ():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_top_route_gb300 import build
    build.build()
    import combine_top_route_gb300 as occ
    occ.lib()
    yield occ
    assert occ.device_error() == 0


def case(T, d, V, dtype="bf16", K=0, ignored=0.0, seed=0, spread=1.8):
    """Inputs on the host: normed rows leaning to their label, a teacher's top tokens."""
    rng = np.random.default_rng(seed + T + d + V)
    w = rng.normal(size=(V, d)).astype(np.float32) * np.float32(spread / d ** 0.5)
    labels = rng.integers(0, V, T).astype(np.int32)
    lean = w[labels] / np.linalg.norm(w[labels], axis=1, keepdims=True)
    x = (rng.normal(size=(T, d)) + 2 * lean).astype(np.float32)
    if dtype == "bf16":
        x, w = (torch.as_tensor(a).bfloat16().float().numpy() for a in (x, w))
    out = rng.random(T) < ignored
    ids = tl = None
    if K:
        ids = rng.integers(0, V, size=(T, K)).astype(np.int32)   # some twice
        ids[:, 0] = labels
        ids[rng.random(T) < 0.2, K // 2 + 1:] = -1
        ids[rng.random(T) < 0.1, 0] = V      # no teacher for these
        tl = (rng.normal(size=(T, K)) * 2 + 5).astype(np.float32)
        tl[rng.random((T, K)) < 0.05] = -np.inf
        ids[out, 0] = -1
    labels[out] = -100
    return x, w, labels, ids, tl


def gpu(a, dt=None):
    if a is None:
        return None
    t = torch.as_tensor(np.ascontiguousarray(a))
    return (t if dt is None else t.to(dt)).cuda()


def run(occ, x, w, labels, ids, tl, dtype="bf16", grad="f32", step=True, want=("dx", "dw"), piece=0,
        tau=1.0, coef=1.0, coef_kd=0.0, coef_z=0.0, dloss=None, stream=None, ws=None):
    T, d = x.shape
    V = len(w)
    K = 0 if ids is None else ids.shape[1]
    cfg = synth.CONFIGS["olmoe_fwd"].with_(T=T, d=d, dtype=dtype)
    ds = occ.desc_for(cfg)
    dt = ds.torch_dtype
    gt = torch.bfloat16 if grad == "bf16" else torch.float32
    opt = occ.occult_head_t(vocab=V, topk=K, grad_dtype=occ.OCCULT_BF16 if grad == "bf16" else occ.OCCULT_F32,
                            piece=piece, coef=coef, coef_kd=coef_kd, coef_z=coef_z, temperature=tau)
    need = occ.head_workspace_size(ds, opt, step=step)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
    new = lambda n, t=torch.float32: torch.full((n + 64,), SENTINEL, dtype=t, device="cuda")  # noqa: E731
    lse, token, loss = new(T), None if labels is None else new(T), new(4)
    kw = dict(labels=gpu(labels), teacher_ids=gpu(ids), teacher_logits=gpu(tl), lse=lse, token_loss=token,
              stream=stream)
    gx, gw = gpu(x, dt), gpu(w, dt)
    dx = dw = None
    torch.cuda.synchronize()
    if step:
        dx, dw = (new(n, gt) if name in want else None for name, n in (("dx", T * d), ("dw", V * d)))
        up = None if dloss is None else torch.full((1,), dloss, device="cuda")
        torch.cuda.synchronize()
        occ.occult_head_step(ds, opt, gx, gw, loss, ws[:need], dx=dx, dw=dw, dloss=up, **kw)
    else:
        occ.occult_head_loss(ds, opt, gx, gw, loss, ws[:need], **kw)
    torch.cuda.synchronize()
    assert (ws[need:] == 255).all()
    out = {}
    for name, t, n in (("loss", loss, 4), ("lse", lse, T), ("token_loss", token, T), ("dx", dx, T * d),
                       ("dw", dw, V * d)):
        if t is not None:
            assert (t[n:] == SENTINEL).all(), name
            out[name] = t[:n].double().cpu().numpy()
            if name in ("dx", "dw"):
                out[name] = out[name].reshape(-1, d)
    return out


def check(occ, c, dtype="bf16", grad="f32", step=True, tau=1.0, coef=1.0, coef_kd=0.0, coef_z=0.0,
          dloss=None, **kw):
    x, w, labels, ids, tl = c
    (T, d), V = x.shape, len(w)
    got = run(occ, *c, dtype=dtype, grad=grad, step=step, tau=tau, coef=coef, coef_kd=coef_kd,
              coef_z=coef_z, dloss=dloss, **kw)
    up = 1.0 if dloss is None else dloss
    clean = np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)
    want = ohead.losses(clean, w, labels, ids, tl, tau=tau, coef=coef, coef_kd=coef_kd, coef_z=coef_z,
                        dloss=up, grads=step)
    x64, w64 = clean.astype(np.float64), w.astype(np.float64)
    bf = dtype == "bf16"
    inside = lambda a: (a >= 0) & (a < V)  # noqa: E731
    ce_on = np.zeros(T, bool) if labels is None else inside(labels)
    kd_on = np.zeros(T, bool) if ids is None else inside(ids[:, 0])
    on = ce_on | kd_on
    mag = np.abs(x64) @ np.abs(w64).T
    ez = ((d / 16 if bf else d) + 8) * 2 * U * mag.max(axis=1)
    e_lse = on * (ez + 300 * U + 4 * U * np.abs(want["lse"]))
    assert (np.abs(got["lse"] - want["lse"]) <= e_lse).all(), np.max(np.abs(got["lse"] - want["lse"]) - e_lse)
    e_tok = e_lse + on * (ez + 4 * U * (np.abs(want["lse"]) + mag.max(axis=1)))
    if labels is not None:
        assert (np.abs(got["token_loss"] - want["token_loss"]) <= e_tok * ce_on).all()
    n_ce, n_kd, n = max(1, ce_on.sum()), max(1, kd_on.sum()), max(1, on.sum())
    red = 40 * U   # the means' trees and the divisions
    e_ce = (e_tok * ce_on).sum() / n_ce + red * want["loss"][1]
    # the terms of kd are of both signs: q (log q - log p), each factor of the size of |log|
    big = 2 * np.abs(tl[np.isfinite(tl)]).max() / tau + 2 * mag.max() / tau + np.log(V) + 40 if ids is not None else 0
    e_kd = tau * tau * ((2 * e_tok / min(1.0, tau) + 160 * U * big) * kd_on).sum() / n_kd
    e_z = (2 * np.abs(want["lse"]) * e_lse).sum() / n + red * want["loss"][3]
    tol = np.array([0, e_ce, e_kd, e_z])
    tol[0] = coef * e_ce + coef_kd * e_kd + coef_z * e_z + 8 * U * (
        coef * want["loss"][1] + coef_kd * np.abs(want["loss"][2]) + coef_z * want["loss"][3])
    assert (np.abs(got["loss"] - want["loss"]) <= tol).all(), (got["loss"], want["loss"], tol)
    if not step:
        return got
    # probabilities of both softmaxes and their errors
    z = x64 @ w64.T
    soft = lambda v: np.exp(v - v.max(axis=1, keepdims=True)) / np.exp(v - v.max(axis=1, keepdims=True)).sum(axis=1, keepdims=True)  # noqa: E731
    p1, p2 = soft(z), soft(z / tau)
    half = max(24.0, 20 * tau) / 65535 * np.log(2) / 2 if bf else 0.0
    floor = 2.0 ** -20 if bf else 0.0
    e1 = ((2 * ez + 700 * U + 8 * U * np.abs(want["lse"]))[:, None] + half) * p1 + floor * p1.max(axis=1, keepdims=True)
    e2 = (((2 * ez + 8 * U * np.abs(want["lse"])) / tau + 700 * U)[:, None] + half / tau) * p2 + floor * p2.max(axis=1, keepdims=True)
    k1 = (ce_on * coef / n_ce + on * 2 * coef_z / n * want["lse"])[:, None]
    has_q = kd_on if ids is None else kd_on & np.array([np.isfinite(tl[t][inside(ids[t])]).any() for t in range(T)])
    k2 = (has_q * coef_kd * tau / n_kd)[:, None]
    dz = k1 * p1 + k2 * p2
    k1e = 2 * coef_z / n * e_lse[:, None]
    pos = np.zeros_like(dz)      # magnitude of what is taken off at the entries
    if labels is not None:
        pos[ce_on, labels[ce_on]] += coef / n_ce
    if ids is not None:
        for t in np.flatnonzero(has_q):
            at = inside(ids[t])
            e = np.exp((tl[t][at].astype(np.float64) - tl[t][at].max()) / tau)
            np.add.at(pos[t], ids[t][at], coef_kd * tau / n_kd * e / e.sum())
    err = k1 * e1 + k2 * e2 + k1e * p1 + 40 * U * (dz + pos)
    if ids is not None:   # the teacher's probabilities: expf and its argument
        err += (2 * np.abs(np.where(np.isfinite(tl), tl, 0)).max() / tau + 20) * U * pos
    size = np.abs(dz - pos)
    if bf:
        err += 2.0 ** -8 * (size + err)
    steps = lambda n_: ((n_ / 16 if bf else n_) + 8) * 2 * U  # noqa: E731
    out_err = 2.0 ** -8 if grad == "bf16" else 2 * U
    for name, a, b, e, k in (("dx", size, w64, err, V), ("dw", size.T, x64, err.T, T)):
        if name not in got:
            continue
        bound = abs(up) * (e @ np.abs(b) + steps(k) * (a @ np.abs(b))) * (1 + 2.0 ** -7) \
            + out_err * np.abs(want[name]) + 1e-36
        off = np.abs(got[name] - want[name])
        assert (off <= bound).all(), (name, np.max(off / bound))
    return got


SIZES = [(1, 64, 16), (1, 2048, 5003), (5, 128, 100), (128, 64, 257), (129, 64, 1000), (257, 192, 777),
         (300, 256, 5000), (513, 320, 2049), (64, 1408, 300), (1, 64, 1), (255, 128, 256), (600, 64, 31)]


@pytest.mark.parametrize("T,d,V", SIZES)
@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_sizes(occ, T, d, V, grad):
    c = case(T, d, V)
    check(occ, c, grad=grad, coef_z=1e-3)
    check(occ, c, step=False, coef_z=1e-3)


@pytest.mark.parametrize("T,d,V", [(1, 4, 3), (7, 64, 1009), (257, 64, 1009), (65, 36, 129), (130, 100, 64)])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("K,tau", [(0, 1.0), (6, 1.5)])
def test_fp32_layers(occ, T, d, V, grad, K, tau):
    c = case(T, d, V, "f32", K=min(K, V), ignored=0.2)
    kw = dict(dtype="f32", coef=0.6, coef_kd=0.5, coef_z=1e-3, tau=tau)
    check(occ, c, grad=grad, dloss=0.5, **kw)
    check(occ, c, step=False, **kw)
    if T > 256:
        check(occ, c, grad=grad, piece=256, **kw)


@pytest.mark.parametrize("K", [1, 5, 33, 64, 128])
@pytest.mark.parametrize("tau", [1.0, 2.0, 0.25, 10.0])
@pytest.mark.parametrize("coef", [0.0, 0.7])
def test_teachers(occ, K, tau, coef):
    """Teacher rows with tokens named twice, out of the vocabulary, at -inf, or none at all."""
    for T, d, V, ignored in ((140, 128, 700, 0.3), (33, 64, 400, 0.0)):
        c = case(T, d, V, K=K, ignored=ignored)
        kw = dict(tau=tau, coef=coef, coef_kd=0.4, coef_z=1e-3 if coef else 0.0)
        check(occ, c, **kw)
        check(occ, c, step=False, **kw)
    x, w, _, ids, tl = c
    tl[:5] = -np.inf
    tl[5:9, 1:] = -np.inf
    check(occ, (x, w, None, ids, tl), tau=tau, coef=0.0, coef_kd=1.0, grad="bf16")


@pytest.mark.parametrize("ignored", [0.0, 0.3, 0.97, 1.0])
@pytest.mark.parametrize("piece", [0, 256])
def test_ignored_rows_and_pieces(occ, ignored, piece):
    """Rows that no term counts may hold anything; a batch in pieces; pieces left empty."""
    for grad in ("f32", "bf16"):
        x, w, labels, ids, tl = case(700, 128, 900, ignored=ignored, seed=3)
        x[labels < 0] = np.nan
        x[np.flatnonzero(labels < 0)[::2]] = np.inf
        check(occ, (x, w, labels, ids, tl), grad=grad, piece=piece, coef_z=1e-3, dloss=-3.0)
        check(occ, (x, w, labels, ids, tl), step=False)


@pytest.mark.parametrize("T,K,ignored", [(3001, 3, 0.4), (2816, 64, 0.0), (3001, 128, 1.0)])
@pytest.mark.parametrize("labelled", [True, False])
def test_many_tokens_with_teachers(occ, T, K, ignored, labelled):
    """So many that rows are counted by tallies of 256 tokens: ends inside one, tokens left out
    on both sides of their borders, labels without a teacher and teachers without a label."""
    x, w, labels, ids, tl = case(T, 64, 300, K=K, ignored=ignored, seed=5)
    labels[::7] = -1
    if ignored < 1:
        labels[250:260], ids[250:260, 0] = -1, -1
    kw = dict(tau=2.0, coef=0.5 if labelled else 0.0, coef_kd=0.5, coef_z=1e-3)
    c = (x, w, labels if labelled else None, ids, tl)
    check(occ, c, piece=1024, **kw)
    check(occ, c, step=False, **kw)


def test_one_gradient_alone(occ):
    c = case(300, 192, 1200, K=8)
    kw = dict(tau=2.0, coef=0.5, coef_kd=0.5)
    both = check(occ, c, **kw)
    for name in ("dx", "dw"):
        got = check(occ, c, want=(name,), **kw)
        assert set(got) == {"loss", "lse", "token_loss", name}
        assert (got[name] == both[name]).all()


def test_large_logits(occ):
    """Logits of thousands: one-hot softmaxes, nothing overflows."""
    for spread in (60.0, 900.0):
        c = case(150, 128, 600, K=7, spread=spread)
        got = check(occ, c, tau=2.0, coef=0.5, coef_kd=0.5)
        assert all(np.isfinite(v).all() for v in got.values())


def test_equal_logits_and_repeats(occ):
    """A zero head; and the same bits from the same call, at any alignment of its tail."""
    x, w, labels, _, _ = case(200, 128, 1000)
    got = check(occ, (x, 0 * w, labels, None, None), coef_z=0.1)
    np.testing.assert_allclose(got["token_loss"], np.log(1000), rtol=1e-6)
    c = case(700, 256, 3001, K=16, ignored=0.2)
    kw = dict(tau=2.0, coef=0.5, coef_kd=0.5, grad="bf16")
    a, b = run(occ, *c, **kw), run(occ, *c, **kw)
    assert all((a[k] == b[k]).all() for k in a)


def test_gradient_is_the_difference_quotient(occ):
    """The kernel's loss of fp32 layers, moved along a random direction of x and of w."""
    c = case(40, 32, 90, "f32", K=5)
    kw = dict(dtype="f32", tau=1.5, coef=0.6, coef_kd=0.5, coef_z=1e-2)
    base = run(occ, *c, **kw)
    rng = np.random.default_rng(1)
    for at, name in ((0, "dx"), (1, "dw")):
        way = rng.normal(size=c[at].shape).astype(np.float32)
        h = 2.0 ** -7
        ends = []
        for sgn in (1, -1):
            cc = list(c)
            cc[at] = c[at] + np.float32(sgn * h) * way
            ends.append(run(occ, *cc, step=False, **kw)["loss"][0])
        num, ana = (ends[0] - ends[1]) / (2 * h), (base[name] * way).sum()
        # the loss is a mean of functions of logits that move by |dz| <= h * s along the way,
        # s their largest speed: third derivatives stay under 4 of it; and fp32's losses
        move = way @ c[1].T if at == 0 else c[0] @ way.T
        s = np.abs(move).max()
        assert abs(num - ana) <= 4 * s ** 3 * h * h / 6 + 64 * U * (abs(ends[0]) + 1) / h


def test_streams_graphs_and_shared_workspaces(occ):
    """A side stream; two graphs over one workspace, replayed in turn on new inputs."""
    T, d, V, K = 300, 128, 1500, 6
    cs = [case(T, d, V, K=K, ignored=0.3, seed=s) for s in (1, 2)]
    kw = dict(tau=2.0, coef=0.5, coef_kd=0.5)
    want = [run(occ, *c, **kw) for c in cs]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = run(occ, *cs[0], stream=s, **kw)
    assert all((got[k] == want[0][k]).all() for k in got)
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, d=d))
    opt = occ.occult_head_t(vocab=V, topk=K, coef=0.5, coef_kd=0.5, temperature=2.0)
    need = max(occ.head_workspace_size(ds, opt, step=b) for b in (True, False))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    x, w = (torch.empty(n, d, dtype=torch.bfloat16, device="cuda") for n in (T, V))
    lab, ids = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, K, dtype=torch.int32, device="cuda")
    tl, lse = torch.empty(T, K, device="cuda"), torch.empty(T, device="cuda")
    loss, dx, dw = torch.empty(2, 4, device="cuda"), torch.empty(T, d, device="cuda"), torch.empty(V, d, device="cuda")

    def fill(c):
        for t, a in zip((x, w, lab, ids, tl), c):
            t.copy_(torch.as_tensor(a))

    fill(cs[0])
    args = dict(labels=lab, teacher_ids=ids, teacher_logits=tl)
    step = lambda: occ.occult_head_step(ds, opt, x, w, loss[0], ws, dx=dx, dw=dw, lse=lse, **args)  # noqa: E731
    only = lambda: occ.occult_head_loss(ds, opt, x, w, loss[1], ws, **args)  # noqa: E731
    step(), only()
    torch.cuda.synchronize()
    graphs = []
    for f in (step, only):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for i in (1, 0, 1):
        fill(cs[i])
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert (dx.double().cpu().numpy() == want[i]["dx"]).all()
        assert (dw.double().cpu().numpy() == want[i]["dw"]).all()
        np.testing.assert_allclose(loss.double().cpu().numpy(), np.tile(want[i]["loss"], (2, 1)), rtol=1e-5)


def test_no_tokens(occ):
    for dtype in ("bf16", "f32"):
        x, w, labels, _, _ = case(3, 64, 50, dtype)
        for grad in ("f32", "bf16"):
            got = run(occ, x[:0], w, labels[:0], None, None, dtype=dtype, grad=grad)
            assert (got["loss"] == 0).all() and (got["dw"] == 0).all()


def test_offsets_past_32_bits(occ):
    """A head of 1.1 million rows of 2048: w and dw hold over 2^31 elements."""
    T, d, V = 3, 2048, 1_100_000
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    for a in range(0, V, 100_000):
        w[a:a + 100_000] = 0.02 * torch.randn(min(100_000, V - a), d, generator=g, device="cuda")
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    labels = torch.tensor([V - 1, 5, V - 700], dtype=torch.int32, device="cuda")
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, d=d))
    opt = occ.occult_head_t(vocab=V, grad_dtype=occ.OCCULT_BF16)
    ws = torch.empty(occ.head_workspace_size(ds, opt), dtype=torch.uint8, device="cuda")
    loss, dx, dw = torch.empty(4, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    occ.occult_head_step(ds, opt, x, w, loss, ws, dx=dx, dw=dw, labels=labels)
    z = torch.cat([x.double() @ w[a:a + 100_000].double().t() for a in range(0, V, 100_000)], dim=1)
    lse = torch.logsumexp(z, dim=1)
    ref = (lse - z[torch.arange(T), labels.long()]).mean()
    # (sums of magnitudes: logits of 2048 products, see above)
    assert abs(float(loss[1]) - float(ref)) < 1e-3
    dz = torch.exp(z - lse[:, None]) / T
    dz[torch.arange(T), labels.long()] -= 1.0 / T
    for rows in (slice(V - 1024, V), slice(0, 64), slice(V // 2, V // 2 + 64)):
        want = dz[:, rows].t() @ x.double()
        size = dz[:, rows].abs().t() @ x.double().abs()
        assert ((dw[rows].double() - want).abs() <= 2.0 ** -6 * size + 1e-9).all()
    want = sum(dz[:, a:a + 100_000] @ w[a:a + 100_000].double() for a in range(0, V, 100_000))
    size = sum(dz[:, a:a + 100_000].abs() @ w[a:a + 100_000].double().abs() for a in range(0, V, 100_000))
    assert ((dx.double() - want).abs() <= 2.0 ** -6 * size).all()


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("d,V", [(64, 1), (64, 3), (2048, 5003), (320, 700), (16384, 130)])
@pytest.mark.parametrize("K,tau", [(0, 1.0), (9, 2.0), (128, 1.0)])
def test_scoring_few_tokens(occ, T, d, V, K, tau):
    c = case(T, d, V, K=K, seed=T)
    check(occ, c, step=False, tau=tau, coef=0.6, coef_kd=0.4, coef_z=1e-3)
    x, w, labels, ids, tl = c
    if T > 1:       # one of them ignored, its row anything
        labels[1] = -1
        x[1] = np.nan
        if K:
            ids[1, 0] = V
        check(occ, c, step=False, tau=tau, coef=0.6, coef_kd=0.4)
    labels[:] = -1
    if K:
        ids[:, 0] = -1
    check(occ, c, step=False, tau=tau, coef=0.6, coef_kd=0.4)


def test_losses_in_pieces(occ):
    """More parts of sums than a workspace of half a GiB holds: the loss goes in pieces."""
    T, d, V = 9000, 64, 750_000
    g = torch.Generator(device="cuda").manual_seed(5)
    w = (1.5 / 8 * torch.randn(V, d, generator=g, device="cuda")).bfloat16()
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    labels = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, d=d))
    opt = occ.occult_head_t(vocab=V)
    need = occ.head_workspace_size(ds, opt, step=False)
    assert need < 1 << 30
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    loss, lse, token = (torch.full((n,), SENTINEL, device="cuda") for n in (4, T, T))
    occ.occult_head_loss(ds, opt, x, w, loss, ws, labels=labels, lse=lse, token_loss=token)
    some = torch.cat([torch.arange(0, T, 211), torch.arange(8160, 8230)]).cuda()
    z = x[some].double() @ w.double().t()
    want = torch.logsumexp(z, dim=1)
    # logits of 64 products: ez = (64 / 16 + 8) 2 u a, a < 64 * 4 * 1.2, and 300 u of the sum
    tol = 12 * 2 * U * 64 * 4 * 1.2 + 300 * U + 4 * U * 20
    assert ((lse[some].double() - want).abs() < tol).all()
    at = z.gather(1, labels[some].long()[:, None])[:, 0]
    assert ((token[some].double() - (want - at)).abs() < 2 * tol).all()
    assert abs(float(loss[1]) - float(token.double().mean())) < 1e-5 * float(loss[1])
    assert abs(float(loss[3]) - float(lse.double().square().mean())) < 1e-5 * float(loss[3])


def test_two_streams_at_once(occ):
    """Two steps over workspaces of their own, on two streams at the same time."""
    T, d, V = 600, 256, 4000
    cs = [case(T, d, V, K=5, ignored=0.2, seed=s) for s in (1, 2)]
    kw = dict(tau=2.0, coef=0.5, coef_kd=0.5)
    want = [run(occ, *c, **kw) for c in cs]
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, d=d))
    opt = occ.occult_head_t(vocab=V, topk=5, coef=0.5, coef_kd=0.5, temperature=2.0)
    streams = [torch.cuda.Stream() for _ in cs]
    args = [dict(x=gpu(c[0], torch.bfloat16), w=gpu(c[1], torch.bfloat16), labels=gpu(c[2]), teacher_ids=gpu(c[3]),
                 teacher_logits=gpu(c[4]), loss=torch.empty(4, device="cuda"),
                 ws=torch.empty(occ.head_workspace_size(ds, opt), dtype=torch.uint8, device="cuda"),
                 dx=torch.empty(T * d, device="cuda"), dw=torch.empty(V * d, device="cuda")) for c in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, a in zip(streams, args):
            occ.occult_head_step(ds, opt, stream=s, **a)
    torch.cuda.synchronize()
    for a, w in zip(args, want):
        assert (a["dx"].view(T, d).double().cpu().numpy() == w["dx"]).all()
        assert (a["dw"].view(V, d).double().cpu().numpy() == w["dw"]).all()


_CAPTURE = """
import sys, torch
sys.path.insert(0, {root!r})
import combine_top_route_gb300 as occ, synth
T, d, V = {T}, 128, 1000
ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, d=d))
opt = occ.occult_head_t(vocab=V)
need = max(occ.head_workspace_size(ds, opt, step=b) for b in (True, False))
ws = torch.empty(need, dtype=torch.uint8, device="cuda")
x, w = torch.randn(T, d, device="cuda").bfloat16(), torch.randn(V, d, device="cuda").bfloat16()
labels = torch.arange(T, device="cuda").int()
loss, dx, dw = torch.empty(2, 4, device="cuda"), torch.empty(T, d, device="cuda"), torch.empty(V, d, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    occ.occult_head_step(ds, opt, x, w, loss[0], ws, dx=dx, dw=dw, labels=labels)
    occ.occult_head_loss(ds, opt, x, w, loss[1], ws, labels=labels)
g.replay()
torch.cuda.synchronize()
a = loss.clone()
occ.occult_head_step(ds, opt, x, w, loss[0], ws, dx=dx, dw=dw, labels=labels)
occ.occult_head_loss(ds, opt, x, w, loss[1], ws, labels=labels)
torch.cuda.synchronize()
assert torch.equal(a, loss) and torch.isfinite(a).all() and abs(float(a[0, 1] - a[1, 1])) < 1e-4, (a, loss)
assert occ.device_error() == 0
print("captured")
"""


@pytest.mark.parametrize("T", [2, 300])
def test_the_first_call_may_be_captured(occ, T):
    """A process whose first call of the head is into a graph."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", _CAPTURE.format(root=root, T=T)], capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0 and "captured" in out.stdout, out.stderr[-2000:]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("taught", [False, True])
def test_tokens_that_are_nearly_sure(occ, dtype, T, taught):
    """1 - p down to 6e-6 of a label's or a teacher's token keeps its digits.

    Every logit is one exact product: a label's of 20 to 32, a rival's g below it, the
    others too low to count, so that a row's sum over its largest term is 1 + e^-g.  What
    is off: the exponential of the largest (2^-22, near 1), the sum's two roundings (2^-24
    each), the probability's exponential (2^-23): 2^-21 in all; the arguments and the
    logarithms, 1e-5 of the result; a bf16 layer's rounding, 2^-8 of it.
    """
    d, V, tau = 64, 1009, 2.0 if taught else 1.0
    j = np.arange(d)
    label, z, g = (37 * j + 5) % V, (160 + 7 * j % 95) / 8, 4.0 + 2 * (j % 5)
    w = np.full((V, d), -512.0, np.float32)
    w[label, j] = z
    w[(label + 500) % V, j] = z - g
    at = np.arange(T) % d
    x = np.zeros((T, d), np.float32)
    x[np.arange(T), at] = 1
    delta = np.exp(-g / tau)                     # a rival's share of its label's
    want, miss = np.log1p(delta)[at], delta / (1 + delta)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, d=d, dtype=dtype))
    opt = occ.occult_head_t(vocab=V, topk=int(taught), coef=1.0 - taught, coef_kd=float(taught), temperature=tau)
    given = dict(labels=gpu(label[at].astype(np.int32)))
    if taught:
        given = dict(teacher_ids=gpu(label[at].astype(np.int32)[:, None]), teacher_logits=torch.zeros(T, 1, device="cuda"))
    xs, ws_ = gpu(x, dt), gpu(w, dt)
    dw = torch.empty(V, d, device="cuda")
    for step in (False, True):
        ws = torch.empty(occ.head_workspace_size(ds, opt, step=step), dtype=torch.uint8, device="cuda")
        loss, tok = torch.empty(4, device="cuda"), torch.empty(T, device="cuda")
        kw = dict(given) if taught else dict(given, token_loss=tok)
        if step:
            occ.occult_head_step(ds, opt, xs, ws_, loss, ws, dw=dw, **kw)
        else:
            occ.occult_head_loss(ds, opt, xs, ws_, loss, ws, **kw)
        if not taught:
            off = np.abs(tok.double().cpu().numpy() - want)
            assert (off <= 2.0 ** -21 + 1e-5 * want).all(), off.max()
        mean = float(loss[2]) / tau ** 2 if taught else float(loss[1])
        assert abs(mean - want.mean()) <= 2.0 ** -21 + 1e-5 * want.mean()
    # a token's gradient at its label, over the tokens that share it
    n = np.bincount(at, minlength=d)
    got = -dw.double().cpu().numpy()[label, j] * T / tau
    tol = n * (2.0 ** -21 + (1e-5 + (2.0 ** -8 if dtype == "bf16" else 0)) * miss)
    assert (np.abs(got - n * miss) <= tol).all(), (np.abs(got - n * miss) / np.maximum(tol, 1e-30)).max()


@pytest.mark.parametrize("tau,taught", [(1.0, False), (1.0, True), (2.0, True), (0.25, True), (10.0, True)])
@pytest.mark.parametrize("V", [300, 1009])
def test_all_gradients_of_sure_tokens(occ, tau, taught, V):
    """Labels (or a teacher's tokens) 12 to 40 octaves, times tau, above every other token: the
    gradients of the others, and so dx, are as small as they are together.

    x picks a column of w each, so that every logit is one exact product and column t of dw is
    the token's dz.  A bf16 layer keeps a step's logits in steps of s = max(24, 20 tau) / 65535
    octaves below the largest of their 128 that is no entry: a probability is within
    s ln 2 / 2 (over tau where tempered) of itself, and one that lies a whole range below, 2^-24
    of that largest's at most (2^-20 tempered), may be 0; one rounding to bf16; sums and
    exponentials 2^-20.
    """
    d, T = 64, 64
    rng = np.random.default_rng(int(10 * tau) + V)
    w = torch.as_tensor(rng.normal(size=(V, d)) * 1.8 * max(1.0, tau ** 0.5)).bfloat16().float().numpy()
    labels = rng.permutation(V)[:T].astype(np.int32)
    up = np.log(2) * (12 + 28 * np.arange(T) / T) * max(1.0, tau)
    w[labels, np.arange(T)] = torch.as_tensor(w.max(axis=0) + up).bfloat16().float().numpy()
    x = np.eye(T, d, dtype=np.float32)
    kw = dict(tau=tau, coef=1.0)
    c = (x, w, labels, None, None)
    K = 0
    if taught:
        K = 3
        ids = rng.integers(0, V, size=(T, K)).astype(np.int32)
        ids[:, 0] = labels
        kw = dict(tau=tau, coef=0.5, coef_kd=0.5)
        c = (x, w, labels, ids, np.array([[9.0, -90.0, -np.inf]] * T, np.float32))
    got = run(occ, *c, **kw)
    want = ohead.losses(*c, **kw)
    p1, p2 = (np.exp(v - v.max(axis=1, keepdims=True)) for v in (w.T.astype(np.float64), w.T / tau))
    p1, p2 = p1 / p1.sum(axis=1, keepdims=True), p2 / p2.sum(axis=1, keepdims=True)
    s = max(24.0, 20 * tau) / 65535 * np.log(2) / 2
    a, b = (0.5 / T, 0.5 * tau / T) if taught else (1.0 / T, 0.0)
    entry = np.zeros((T, V), bool)
    entry[np.arange(T), labels] = True
    if taught:
        entry[np.arange(T)[:, None], ids] = True
    err = np.zeros((T, V))
    for c0 in range(0, V, 128):
        part = slice(c0, min(V, c0 + 128))
        top1, top2 = (np.where(entry, 0, p)[:, part].max(axis=1, keepdims=True) for p in (p1, p2))
        reach = max(24.0, 20 * tau)
        err[:, part] = a * (s * p1[:, part] + 2.0 ** -reach * top1) + b * (s / tau * p2[:, part] + 2.0 ** (-reach / tau) * top2)
    # an entry's own is of the size of what all others are together
    miss = a * (np.where(entry, 0, p1).sum(axis=1, keepdims=True)) + b * (np.where(entry, 0, p2).sum(axis=1, keepdims=True))
    size = a * p1 + b * p2
    err = np.where(entry, 2.0 ** -20 * (miss + a + b), err + 2.0 ** -20 * size)
    exact = want["dw"].T[:T]                     # dz [T, V]
    err = err + 2.0 ** -8 * (np.abs(exact) + err)
    off = np.abs(got["dw"].T[:T] - exact)
    assert (off <= err * (1 + 2.0 ** -10)).all(), np.max(off / err)
    bound = err @ np.abs(w) + (V / 16 + 8) * 2 * U * (np.abs(exact) @ np.abs(w))
    off = np.abs(got["dx"] - want["dx"])
    assert (off <= bound * (1 + 2.0 ** -7)).all(), np.max(off / bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("coefs", [(1e-42, 0.7, 1e-2), (1e-38, 0.0, 1e-2), (0.0, 1e-40, 1.0), (1e28, 1e-12, 0.0)])
def test_terms_of_far_apart_weights(occ, dtype, coefs):
    """A term that weighs next to nothing leaves the others' gradients as they are alone."""
    coef, coef_kd, coef_z = coefs
    c = case(200, 128, 700, dtype, K=4, ignored=0.2)
    kw = dict(dtype=dtype, tau=2.0)
    big = dict(coef=coef if coef > 1e-20 else 0.0, coef_kd=coef_kd if coef_kd > 1e-5 else 0.0, coef_z=coef_z)
    got = run(occ, *c, coef=coef, coef_kd=coef_kd, coef_z=coef_z, **kw)
    alone = run(occ, *c, **big, **kw)
    for name in ("dx", "dw"):
        assert np.isfinite(got[name]).all()
        # (the common factor differs: dz is rounded to bf16 at another place, once each)
        tol = (2.0 ** -7 if dtype == "bf16" else 2.0 ** -20)
        assert np.linalg.norm(got[name] - alone[name]) <= tol * np.linalg.norm(alone[name])


def bf16(v):
    return torch.as_tensor(v, dtype=torch.float64).float().bfloat16().double().numpy()


@pytest.mark.parametrize("case_", ["few", "pieces", "taught"])
def test_entries_gradients_lose_half_a_unit_at_most_where_it_is_small(occ, case_):
    """A piece whose entries' gradients all have one size is rounded where half a unit is least of it.

    Half a unit of bf16 is 2^-8 of a number just above a power of two and 2^-9 of one just below.
    Some stretch 2^(j / 8) of the eight takes any number to a fraction of 2^(7 / 8) and more, so
    that the least error is at most 2^-8 / 2^(7 / 8) = 0.00213 of it, and the exponentials' 2^-19.
    The sizes here are those that lose the most as they are.  x picks a column of w, so that a
    column of dw is the pieces' dz, over tokens of one dz each.
    """
    d, V = 64, 5
    tau = 2.0 if case_ == "taught" else 1.0
    # labels' logits above four others at 0: 1 - p of them, by what bf16 takes from it
    z = bf16(np.linspace(0.5, 6.0, 3000))
    miss = 4 / (4 + np.exp(z / tau))
    loss = np.abs(bf16(miss) - miss) / miss
    worst = z[np.argsort(-loss)[:64]]
    assert np.sort(loss)[-64:].min() > 0.0025   # (the inputs alone, before any call)
    w = np.zeros((V, d), np.float32)
    w[0] = worst
    calls = [(np.full(n, i), 0) for i in range(64) for n in (1, 3)] if case_ != "pieces" else [
        (np.repeat([i, i + 1, i + 2], [256, 256, 90]), 256) for i in range(0, 60, 12)]
    for cols, piece in calls:
        T = len(cols)
        x = np.zeros((T, d), np.float32)
        x[np.arange(T), cols] = 1
        lab = np.zeros(T, np.int32)
        kw = dict(piece=piece, tau=tau)
        if case_ == "taught":
            got = run(occ, x, w, None, lab[:, None], np.zeros((T, 1), np.float32), coef=0.0, coef_kd=1.0, **kw)
        else:
            got = run(occ, x, w, lab, None, None, **kw)
        for c in np.unique(cols):
            want = -(cols == c).sum() / T * tau * 4 / (4 + np.exp(float(w[0, c]) / tau))
            assert abs(got["dw"][0, c] / want - 1) <= 2.0 ** -8 / 2 ** (7 / 8) + 2.0 ** -19 + 2 * U * T


@pytest.mark.parametrize("T,step", [(1, True), (5, False), (128, False), (128, True)])
@pytest.mark.parametrize("d", [512, 2048])
def test_logits_of_few_tokens_lose_a_segment_at_most(occ, T, step, d):
    """Sums that the tensor cores truncate at every step: 256 products to a segment.

    The first of a logit's products is 1, and every further 16 of them add up to a little
    less than fp32's step above 1: one of the tensor cores' steps each, dropped.  A segment of
    256 has 16 steps and the later ones have no large term, so that less than 16 * 2^-23 is
    lost; joining up to eight segments rounds to nearest (2^-24 each), the log-sum of the one
    logit is its product with log2(e) and back, three roundings of 2^-24 of 1.5.
    """
    x = np.ones((T, d), np.float32)
    w = np.full((1, d), 127 / 128 * 2.0 ** -27, np.float32)
    w[0, :16] = 0
    w[0, 0] = 1
    want = 1 + (d / 16 - 1) * 127 / 128 * 2.0 ** -23
    got = run(occ, x, w, np.zeros(T, np.int32), None, None, step=step)
    assert np.abs(got["lse"] - want).max() <= 16 * 2.0 ** -23 + 8 * U + 3 * 1.5 * U
