"""GPU parity of occult_balance_loss and occult_balance_grad with the fp64 oracle.

Counts are exact.  With u = 2^-24: a probability (expf 2 units, the argument's
rounding up to 20 u, a sum of 256 terms as a tree of 8 + 8, a division) is within
P = 64 u of itself; the sums over tokens and experts are of positive terms in chains
of at most 1024 additions, so a loss term is within SUM = 1100 u of itself.  The
gradient's weights are within SUM' = 16 u of themselves (counts are exact).
"""
import numpy as np
import pytest
import torch

import synth
from oracle import balance as obal

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
P, SUM = 64 * U, 1100 * U
COEF = dict(coef=0.3, coef_dev=0.2, coef_z=0.1)


@pytest.fixture(scope="module")
def occ():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_top_route_gb300 import build
    build.build()
    import combine_top_route_gb300 as occ
    occ.lib()
    return occ


def case(T, Ne, k, seed=0):
    rng = np.random.default_rng(seed)
    boost = rng.random((8, Ne)) < 0.2
    z = (rng.normal(size=(T, Ne)) + 3.0 * boost[rng.integers(0, 8, T)]).astype(np.float32)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    return z, ids


def run(occ, z, ids, e2v, Nd, group_len=0, mask=None, base=None, dloss=None, stream=None):
    T, Ne = z.shape
    k = ids.shape[1]
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, n_experts=Ne, top_k=k, n_vdev=Nd))
    opt = occ.occult_balance_t(COEF["coef"], COEF["coef_dev"], COEF["coef_z"], group_len)
    G = occ.balance_groups(ds, opt)
    c = lambda a, dt: None if a is None else torch.as_tensor(np.ascontiguousarray(a)).to(dt).cuda()  # noqa: E731
    counts = torch.full((G * Ne + 8,), -7, dtype=torch.int32, device="cuda")
    grad_w = torch.full((G * Ne + 1 + 8,), -7.0, device="cuda")
    loss = torch.full((4 + 4,), -7.0, device="cuda")
    ws = torch.full((occ.balance_workspace_size(ds, opt),), 255, dtype=torch.uint8, device="cuda")
    logits, m = c(z, torch.float32), c(mask, torch.uint8)
    dl = torch.full((T * Ne + 8,), -7.0, device="cuda")
    if base is not None:
        dl[:T * Ne] = c(base, torch.float32).view(-1)
    up = None if dloss is None else torch.full((1,), dloss, device="cuda")
    occ.occult_balance_loss(ds, opt, logits, c(ids, torch.int32), c(e2v, torch.int32), counts,
                            grad_w, loss, ws, mask=m, stream=stream)
    occ.occult_balance_grad(ds, opt, logits, grad_w, dl, mask=m, dloss=up,
                            accumulate=base is not None, stream=stream)
    torch.cuda.synchronize()
    assert (counts[G * Ne:] == -7).all() and (grad_w[G * Ne + 1:] == -7).all()
    assert (loss[4:] == -7).all() and (dl[T * Ne:] == -7).all()
    return (loss[:4].double().cpu().numpy(), counts[:G * Ne].cpu().numpy().reshape(G, Ne),
            dl[:T * Ne].double().cpu().numpy().reshape(T, Ne))


def check(occ, z, ids, Nd, group_len=0, mask=None, base=None, dloss=None, seed=1, **kw):
    Ne = z.shape[1]
    e2v = np.random.default_rng(seed).permutation(Ne) % Nd
    got = run(occ, z, ids, e2v, Nd, group_len, mask, base, dloss, **kw)
    loss, counts, grad = obal.loss_and_grad(z, ids, e2v, Nd, group_len, mask, **COEF)
    assert (got[1] == counts).all()
    # z squares a logarithm: its relative error is twice that of lse, which a cancellation
    # max + log(sum) can make larger than P (of the magnitude of the parts)
    live = np.ones(len(z), bool) if mask is None else np.asarray(mask, bool)
    lse = np.zeros(len(z))
    top = np.zeros(len(z))
    if live.any():
        zz = z[live].astype(np.float64)
        top[live] = zz.max(axis=1)
        lse[live] = top[live] + np.log(np.exp(zz - top[live][:, None]).sum(axis=1))
    e_lse = 8 * U * (np.abs(top) + 8) + P
    n = max(1, live.sum())
    e_z = (2 * np.abs(lse) * e_lse * live).sum() / n + SUM * loss[3]
    tol = np.array([0, SUM * loss[1], SUM * loss[2], e_z])
    tol[0] = abs(COEF["coef"]) * tol[1] + COEF["coef_dev"] * tol[2] + COEF["coef_z"] * tol[3] \
        + 4 * U * abs(loss[0])
    assert (np.abs(got[0] - loss) <= tol).all(), (got[0], loss, tol)
    # the gradient: p (w - w.p) + wz lse p, each factor's error
    p = np.zeros_like(z, dtype=np.float64)
    p[live] = np.exp(z[live].astype(np.float64) - lse[live][:, None])
    groups = obal.groups(len(z), group_len)
    wmax = np.zeros(len(z))
    for gi, g in enumerate(groups):
        N = live[list(g)].sum() if len(g) else 0
        if N:
            f = counts[gi] * Ne / (ids.shape[1] * N)
            A = max(1, sum(1 for h in groups if live[list(h)].any()))
            fd = np.array([f[e2v == e2v[e]].mean() for e in range(Ne)])
            wmax[list(g)] = (COEF["coef"] * f + COEF["coef_dev"] * fd).max() / (A * N)
    up = 1.0 if dloss is None else dloss
    wz = 2 * COEF["coef_z"] / n
    err = p * (2 * wmax * (2 * P + 32 * U) + wz * (np.abs(lse) * (P + 8 * U) + e_lse))[:, None]
    want = up * grad + (0 if base is None else base)
    err = abs(up) * err + 3 * U * (np.abs(want) + (0 if base is None else np.abs(base))) + 1e-37
    bad = np.abs(got[2] - want) - err
    assert bad.max() <= 0, (np.unravel_index(bad.argmax(), bad.shape), bad.max())


@pytest.mark.parametrize("T,Ne,k,Nd", [(1, 8, 2, 4), (7, 8, 2, 4), (256, 8, 2, 4), (300, 60, 4, 4),
                                       (1000, 64, 8, 8), (513, 33, 3, 1), (129, 96, 12, 32),
                                       (700, 128, 16, 16), (333, 256, 8, 32), (64, 1, 1, 1),
                                       (50, 2, 2, 2), (4100, 64, 6, 8), (90, 255, 5, 5),
                                       (257, 64, 4, 8), (8192, 64, 2, 8), (8193, 64, 2, 8),
                                       (65, 256, 8, 8), (2048, 256, 2, 8), (2049, 256, 2, 8)])
def test_sizes(occ, T, Ne, k, Nd):
    z, ids = case(T, Ne, k, seed=T)
    check(occ, z, ids, Nd)


@pytest.mark.parametrize("group_len", [1, 7, 64, 100, 128, 999, 1000, 4096])
@pytest.mark.parametrize("Ne", [8, 64, 160])
def test_groups_and_masks(occ, group_len, Ne):
    """Ragged last groups, groups without a token, NaN and infinity under the mask."""
    T = 1000 if group_len > 1 else 60
    z, ids = case(T, Ne, 4, seed=group_len)
    rng = np.random.default_rng(2)
    mask = rng.random(T) < 0.7
    mask[: min(group_len, T // 2)] = False                 # the first group is empty
    z[~mask] = rng.choice([np.nan, np.inf, -np.inf, 3e38], size=((~mask).sum(), 1))
    ids[~mask] = rng.integers(-2**31, 2**31 - 1, size=((~mask).sum(), 4))
    check(occ, z, ids, 4, group_len, mask)
    check(occ, z, ids, 8, group_len, mask, base=rng.normal(size=z.shape).astype(np.float32), dloss=-2.5)


def test_every_token_masked(occ):
    z, ids = case(70, 16, 2)
    z[:] = np.nan
    loss, counts, grad = run(occ, z, ids, np.arange(16) % 4, 4, 32, np.zeros(70))
    assert not loss.any() and not counts.any() and not grad.any()


def test_masked_tokens_keep_what_is_accumulated(occ):
    z, ids = case(40, 16, 2)
    mask = np.arange(40) % 2
    base = np.random.default_rng(0).normal(size=z.shape).astype(np.float32)
    _, _, grad = run(occ, z, ids, np.arange(16) % 4, 4, 0, mask, base)
    assert (grad[mask == 0] == base[mask == 0]).all()


def test_dropped_slots_and_masked_experts(occ):
    """Ids outside the experts count nothing; logits of -inf have no probability and no
    gradient (the lowest finite value likewise)."""
    z, ids = case(200, 64, 4, seed=11)
    ids[::3, 3] = -1
    ids[1::3, 2] = 64
    z[:, 5] = -np.inf
    z[:, 6] = np.finfo(np.float32).min
    z[:100, 32:] = -np.inf
    ids = np.where((ids >= 32) | (ids == 5) | (ids == 6), -1, ids).astype(np.int32)
    check(occ, z, ids, 8)


def test_large_and_negative_logits(occ):
    z, ids = case(100, 64, 4, seed=12)
    check(occ, (z - 80).astype(np.float32), ids, 8)
    check(occ, (z * 3 + 80).astype(np.float32), ids, 8)


def test_no_tokens(occ):
    loss, counts, grad = run(occ, np.zeros((0, 16), np.float32), np.zeros((0, 2), np.int32),
                             np.arange(16) % 4, 4)
    assert not loss.any() and counts.shape == (1, 16) and not counts.any()


def test_bit_reproducible_and_on_a_side_stream(occ):
    z, ids = case(3000, 64, 8, seed=13)
    e2v = np.arange(64) % 8
    s = torch.cuda.Stream()
    a = run(occ, z, ids, e2v, 8, 500)
    for _ in range(3):
        torch.cuda.synchronize()
        b = run(occ, z, ids, e2v, 8, 500, stream=s)
        assert all((x == y).all() for x, y in zip(a, b))


def test_large_batch_against_doubles(occ):
    """131072 tokens of 256 experts in 32 groups, masked, against fp64 on the GPU."""
    T, Ne, k, L = 131072, 256, 8, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn(T, Ne, generator=g, device="cuda")
    ids = z.topk(k, dim=1).indices.to(torch.int32).contiguous()
    mask = (torch.rand(T, generator=g, device="cuda") < 0.9).to(torch.uint8)
    mask[-L:] = 0
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, n_experts=Ne, top_k=k, n_vdev=8))
    opt = occ.occult_balance_t(1.0, 0.0, 0.0, L)
    G = occ.balance_groups(ds, opt)
    counts = torch.empty(G, Ne, dtype=torch.int32, device="cuda")
    grad_w, loss = torch.empty(G * Ne + 1, device="cuda"), torch.empty(4, device="cuda")
    ws = torch.empty(occ.balance_workspace_size(ds, opt), dtype=torch.uint8, device="cuda")
    e2v = (torch.arange(Ne, device="cuda") % 8).to(torch.int32)
    dl = torch.empty(T, Ne, device="cuda")
    occ.occult_balance_loss(ds, opt, z, ids, e2v, counts, grad_w, loss, ws, mask=mask)
    occ.occult_balance_grad(ds, opt, z, grad_w, dl, mask=mask)
    p = z.double().softmax(1) * mask[:, None]
    one = torch.nn.functional.one_hot(ids.long(), Ne).sum(1) * mask[:, None]
    want = one.view(G, L, Ne).sum(1)
    assert torch.equal(counts.long(), want)
    N = mask.view(G, L).sum(1).double()
    f = want * Ne / (k * N.clamp(min=1)[:, None])
    S = p.view(G, L, Ne).sum(1) / N.clamp(min=1)[:, None]
    bal = float((f * S).sum() / (G - 1))
    assert abs(float(loss[1]) - bal) <= 1100 * U * bal
    w = (f / ((G - 1) * N.clamp(min=1))[:, None]).repeat_interleave(L, 0)
    dz = p * (w - (p * w).sum(1, keepdim=True))
    err = (p * w.amax(1, keepdim=True)) * (2 * (2 * P + 32 * U)) + 3 * U * dz.abs() + 1e-37
    assert ((dl.double() - dz).abs() <= err).all()


def test_more_groups_than_a_grid_has_rows(occ):
    """70000 sequences of one token, every third masked, against fp64 on the GPU."""
    T, Ne, k = 70000, 8, 2
    g = torch.Generator(device="cuda").manual_seed(4)
    z = torch.randn(T, Ne, generator=g, device="cuda")
    ids = z.topk(k, dim=1).indices.to(torch.int32).contiguous()
    mask = (torch.arange(T, device="cuda") % 3 != 0).to(torch.uint8)
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, n_experts=Ne, top_k=k, n_vdev=4))
    opt = occ.occult_balance_t(1.0, 0.0, 0.5, 1)
    assert occ.balance_groups(ds, opt) == T
    counts = torch.empty(T, Ne, dtype=torch.int32, device="cuda")
    grad_w, loss = torch.empty(T * Ne + 1, device="cuda"), torch.empty(4, device="cuda")
    ws = torch.empty(occ.balance_workspace_size(ds, opt), dtype=torch.uint8, device="cuda")
    e2v = (torch.arange(Ne, device="cuda") % 4).to(torch.int32)
    occ.occult_balance_loss(ds, opt, z, ids, e2v, counts, grad_w, loss, ws, mask=mask)
    on = mask.double()[:, None]
    one = torch.nn.functional.one_hot(ids.long(), Ne).sum(1) * mask[:, None]
    assert torch.equal(counts.long(), one)
    p, lse = z.double().softmax(1), z.double().logsumexp(1)
    bal = float((one * (Ne / k) * p * on).sum() / on.sum())
    sq = float((lse.square() * on[:, 0]).sum() / on.sum())
    assert abs(float(loss[1]) - bal) <= SUM * bal and abs(float(loss[3]) - sq) <= SUM * sq


@pytest.mark.parametrize("T,group_len", [(70000, 0), (5000, 1300)])
@pytest.mark.parametrize("Ne,k", [(1, 1), (5, 2), (8, 2), (7, 7), (8, 5), (13, 2), (16, 4), (16, 16),
                                  (20, 3), (31, 8), (32, 8), (33, 8), (37, 16), (100, 6), (130, 1),
                                  (255, 16)])
def test_every_number_of_lanes(occ, Ne, k, T, group_len):
    """Experts and slots around what one to 32 lanes a token hold, whole rows of 16-byte
    words and others, in two launches."""
    z, ids = case(T, Ne, k, seed=Ne + k)
    mask = np.random.default_rng(3).random(T) < 0.8
    check(occ, z, ids, 1, group_len, mask)


@pytest.mark.parametrize("Ne", [8, 64, 160])
@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("group_len", [0, 300])
def test_weights_of_one_layer_of_several(occ, Ne, off, group_len):
    """grad_w rows of a buffer of several layers' (G Ne + 1 words each) begin at no whole 16
    bytes; loss and gradient take them alike, with the gradient of an aligned buffer but
    for the order of one sum."""
    T, k = 1000, 2
    z, ids = case(T, Ne, k, seed=Ne)
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, n_experts=Ne, top_k=k, n_vdev=4))
    opt = occ.occult_balance_t(COEF["coef"], COEF["coef_dev"], COEF["coef_z"], group_len)
    n = occ.balance_groups(ds, opt) * Ne + 1
    z, ids = torch.as_tensor(z).cuda(), torch.as_tensor(ids).cuda()
    e2v = (torch.arange(Ne, device="cuda") % 4).to(torch.int32)
    counts, loss = torch.empty((n - 1,), dtype=torch.int32, device="cuda"), torch.empty(4, device="cuda")
    ws = torch.empty(occ.balance_workspace_size(ds, opt), dtype=torch.uint8, device="cuda")
    grads = []
    for o in (0, off):
        grad_w = torch.full((n + 8,), -7.0, device="cuda")
        view = grad_w[o:o + n]
        dl = torch.empty(T, Ne, device="cuda")
        occ.occult_balance_loss(ds, opt, z, ids, e2v, counts, view, loss, ws)
        occ.occult_balance_grad(ds, opt, z, view, dl)
        assert (grad_w[:o] == -7).all() and (grad_w[o + n:] == -7).all()
        grads.append((view.clone(), dl.double()))
    (wa, a), (wb, b) = grads
    assert torch.equal(wa, wb)
    # p (w - w.p + wz lse): two orders of a sum of Ne positive terms, within 32 units of w
    # for a factor of p, and the units of the products
    p = z.double().softmax(1)
    w = wa[:-1].double().view(-1, Ne).repeat_interleave(group_len or T, 0)[:T]
    err = p * (32 * U * w.amax(1, keepdim=True)) + 4 * U * a.abs()
    assert ((a - b).abs() <= err + 1e-37).all()
