"""GPU parity of occult_block_norm and occult_block_norm_bwd with the fp64 oracle.

Tolerances, element by element, with u = 2^-24: sums over a row run as chains of at
most CHAIN fp32 additions (a thread's own elements, then a tree), so a mean square
is within CHAIN u of itself relatively and 1 / sqrt of it within half that plus
rsqrtf's 2 units; products and sums of a few terms add single units of the terms'
magnitudes; rounding to bf16 adds 2^-8, to fp32 2^-24 of the result.  Column sums
over the tokens run as at most COLS additions.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import block_norm as onorm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CHAIN = 96
RSTD = (CHAIN / 2 + 6) * U
COLS = 1024
EPS = 1e-5
UNIT = {"bf16": 2.0 ** -8, "f32": U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 64  # elements after every output that must stay as they were


@pytest.fixture(scope="module")
def occ():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_top_route_gb300 import build
    build.build()
    import combine_top_route_gb300 as occ
    occ.lib()
    return occ


def rounded(a, kind):
    """fp64 array of values that the type holds."""
    return torch.as_tensor(a, dtype=torch.float32).to(DT[kind]).double().numpy()


class Case:
    def __init__(self, T, d, dtype, res, post=True, pre=True, gate="none", y=True, seed=0,
                 res_scale=0.75):
        rng = np.random.default_rng(seed)
        self.T, self.d, self.dtype, self.res, self.gate = T, d, dtype, res, gate
        self.res_scale = res_scale
        n = lambda *s: rng.normal(size=s)  # noqa: E731
        self.r = rounded(2 * n(T, d), res)
        self.y = rounded(n(T, d), "f32") if y else None
        self.w_post = rounded(1 + 0.3 * n(d), dtype) if post else None
        self.w_pre = rounded(1 + 0.3 * n(d), dtype) if pre else None
        self.g = {"none": None, "channel": rounded(n(d), "f32"),
                  "token": rounded(n(T, 1), "f32")}[gate]
        self.dr_out, self.dx = rounded(n(T, d), res), rounded(n(T, d), "f32")

    def desc(self, occ):
        cfg = synth.CONFIGS["olmoe_fwd"].with_(T=self.T, d=self.d, dtype=self.dtype, inter=64)
        return occ.desc_for(cfg)

    def opt(self, occ):
        kind = {"none": occ.GATE_NONE, "channel": occ.GATE_CHANNEL, "token": occ.GATE_TOKEN}
        return occ.occult_norm_t(EPS, self.res_scale, kind[self.gate],
                                 occ.OCCULT_BF16 if self.res == "bf16" else occ.OCCULT_F32)


def dev(a, kind):
    return None if a is None else torch.as_tensor(a).to(DT[kind]).cuda().contiguous()


def out(n, kind):
    return torch.full((n + GUARD,), 77.0, dtype=DT[kind], device="cuda")


def take(t, shape):
    """The output's values; checks that nothing was written past it."""
    n = int(np.prod(shape))
    assert (t[n:] == 77.0).all()
    return t[:n].double().cpu().numpy().reshape(shape)


def close(got, want, tol, what):
    assert np.isfinite(got).all() and got.shape == want.shape, what
    if not got.size:
        return
    bad = np.abs(got - want) - tol
    i = np.unravel_index(np.argmax(bad), bad.shape)
    assert bad[i] <= 0, f"{what}{list(i)}: {got[i]} against {want[i]}, tolerance {np.broadcast_to(tol, bad.shape)[i]}"


def run_forward(occ, c, inplace=False, stream=None):
    T, d = c.T, c.d
    r = dev(c.r, c.res)
    r_out = None
    if c.y is not None:
        if inplace:
            r_out = out(T * d, c.res)
            r_out[:T * d] = r.view(-1)
            r = r_out
        else:
            r_out = out(T * d, c.res)
    x = out(T * d, c.dtype) if c.w_pre is not None else None
    rp = out(T, "f32") if c.w_post is not None else None
    rq = out(T, "f32") if c.w_pre is not None else None
    occ.occult_block_norm(c.desc(occ), c.opt(occ), r, y=dev(c.y, "f32"),
                          w_post=dev(c.w_post, c.dtype), gate=dev(c.g, "f32"),
                          w_pre=dev(c.w_pre, c.dtype), r_out=r_out, x=x, rstd_post=rp,
                          rstd_pre=rq, stream=stream)
    torch.cuda.synchronize()
    return r_out, x, rp, rq


def check_forward(occ, c, **kw):
    r_out, x, rp, rq = run_forward(occ, c, **kw)
    want = onorm.forward(c.r, c.y, c.w_post, c.g, c.w_pre, EPS, c.res_scale)
    T, d = c.T, c.d
    s, e_s = c.r, np.zeros((T, d))
    if rp is not None:
        close(take(rp, (T,)), want["rstd_post"], RSTD * want["rstd_post"], "rstd_post")
    if r_out is not None:
        s = want["r_out"]
        b = s - c.res_scale * c.r
        e_s = (8 * U + RSTD) * (np.abs(c.res_scale * c.r) + np.abs(b))
        close(take(r_out, (T, d)), s, e_s + UNIT[c.res] * (np.abs(s) + e_s), "r_out")
    if x is not None:
        q = want["rstd_pre"]
        ss = (s * s).sum(axis=1)
        e_q = RSTD + np.where(ss > 0, (np.abs(s) * e_s).sum(axis=1) / np.where(ss > 0, ss, 1), 0)
        close(take(rq, (T,)), q, e_q * q, "rstd_pre")
        e = (e_s * q[:, None] + np.abs(s) * (q * (e_q + 4 * U))[:, None]) * np.abs(c.w_pre)
        close(take(x, (T, d)), want["x"], e + UNIT[c.dtype] * (np.abs(want["x"]) + e), "x")


def check_backward(occ, c, dr_out=True, inplace=False):
    T, d = c.T, c.d
    fw = onorm.forward(c.r, c.y, c.w_post, c.g, c.w_pre, EPS, c.res_scale)
    saved = rounded(fw["r_out"], c.res) if c.y is not None else c.r
    rp = rounded(fw["rstd_post"], "f32") if c.w_post is not None else None
    rq = rounded(fw["rstd_pre"], "f32") if c.w_pre is not None else None
    up_r = c.dr_out if dr_out else None
    up_x = c.dx if c.w_pre is not None else None
    want = onorm.backward(up_r, up_x, saved, c.y, c.w_post, c.g, c.w_pre, rp, rq, c.res_scale)
    dr = out(T * d, c.res)
    src = dev(up_r, c.res)
    if inplace:
        dr[:T * d] = src.view(-1)
        src = dr
    o = {"dr": dr, "dy": out(T * d, c.dtype) if c.y is not None else None,
         "dw_post": out(d, "f32") if c.w_post is not None else None,
         "dw_pre": out(d, "f32") if c.w_pre is not None else None,
         "dgate": None if c.g is None else out(c.g.size, "f32")}
    ds = c.desc(occ)
    ws = torch.full((occ.workspace_size(ds, occ.WS_BLOCK_NORM_BWD),), 255, dtype=torch.uint8,
                    device="cuda")
    occ.occult_block_norm_bwd(ds, c.opt(occ), src, dev(saved, c.res), o["dr"], ws,
                              dx=dev(up_x, "f32"), y=dev(c.y, "f32"),
                              w_post=dev(c.w_post, c.dtype), gate=dev(c.g, "f32"),
                              w_pre=dev(c.w_pre, c.dtype), rstd_post=dev(rp, "f32"),
                              rstd_pre=dev(rq, "f32"), dy=o["dy"], dw_post=o["dw_post"],
                              dgate=o["dgate"], dw_pre=o["dw_pre"])
    torch.cuda.synchronize()
    assert set(want) == {k for k, v in o.items() if v is not None}
    # error of D
    D0, e_D = np.zeros((T, d)) if up_r is None else np.abs(up_r), 0.0
    e_c1 = np.zeros((T, 1))
    n = np.zeros((T, d))
    D = np.zeros((T, d)) if up_r is None else up_r
    if c.w_pre is not None:
        n = saved * rq[:, None]
        g = up_x * c.w_pre
        c1 = (g * n).mean(axis=1, keepdims=True)
        e_c1 = (CHAIN + 4) * U * np.abs(g * n).mean(axis=1, keepdims=True)
        D = D + rq[:, None] * (g - n * c1)
        mag = D0 + rq[:, None] * (np.abs(g) + np.abs(n * c1))
        e_D = 8 * U * mag + rq[:, None] * np.abs(n) * e_c1
        D0 = mag
        close(take(o["dw_pre"], (d,)), want["dw_pre"], COLS * U * np.abs(up_x * n).sum(axis=0), "dw_pre")
    a = c.res_scale if c.y is not None else 1.0
    e = abs(a) * e_D + 2 * U * np.abs(want["dr"])
    close(take(o["dr"], (T, d)), want["dr"], e + UNIT[c.res] * (np.abs(want["dr"]) + e), "dr")
    if c.y is None:
        return
    m = c.y if rp is None else c.y * rp[:, None]
    b = m if c.w_post is None else m * c.w_post
    gate = np.ones((1, 1)) if c.g is None else c.g
    # a sum over a row of D b: every term's D error, the chain's, the mean's
    e_row = (np.abs(b) * (e_D + 8 * U * D0)).sum(axis=1, keepdims=True) \
        + (CHAIN + 8) * U * (np.abs(b) * (D0 + np.abs(n))).sum(axis=1, keepdims=True)
    if c.gate == "token":
        close(take(o["dgate"], (T,)), want["dgate"], e_row[:, 0], "dgate")
    cols = lambda v: COLS * U * np.abs(v).sum(axis=0)  # noqa: E731
    if c.gate == "channel":
        close(take(o["dgate"], (d,)), want["dgate"],
              (np.abs(b) * e_D).sum(axis=0) + cols(D0 * b), "dgate")
    u = gate * D
    e_u = np.abs(gate) * e_D + 2 * U * np.abs(u)
    if c.w_post is not None:
        close(take(o["dw_post"], (d,)), want["dw_post"],
              (np.abs(m) * e_u).sum(axis=0) + cols(np.abs(gate) * D0 * m), "dw_post")
        uw = u * c.w_post
        gm = np.abs(gate) if c.gate != "token" else np.abs(c.g)
        bg = np.abs(b) * (np.abs(gate) if c.gate == "channel" else 1.0)
        e_c2 = ((bg * (e_D + 8 * U * D0)).sum(axis=1, keepdims=True)
                + (CHAIN + 8) * U * (bg * (D0 + np.abs(n))).sum(axis=1, keepdims=True)) \
            * (gm if c.gate == "token" else 1.0) / d
        c2 = (uw * m).mean(axis=1, keepdims=True)
        e_u = rp[:, None] * (e_u * np.abs(c.w_post) + 4 * U * np.abs(uw)
                             + np.abs(m) * (e_c2 + 4 * U * np.abs(c2)))
    close(take(o["dy"], (T, d)), want["dy"],
          e_u + UNIT[c.dtype] * (np.abs(want["dy"]) + e_u), "dy")


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")]
SIZES = [(1, 64), (1, 2048), (2, 64), (33, 128), (257, 64), (300, 192), (129, 320), (64, 512),
         (97, 1024), (31, 1408), (513, 2048), (19, 2112), (41, 4096), (7, 5632), (5, 8192),
         (3, 16384)]


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("T,d", SIZES)
def test_forward_sizes(occ, T, d, dtype, res):
    check_forward(occ, Case(T, d, dtype, res, gate="channel", seed=T + d))


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("T,d", SIZES)
def test_backward_sizes(occ, T, d, dtype, res):
    check_backward(occ, Case(T, d, dtype, res, gate="channel", seed=T + d))


@pytest.mark.parametrize("d", [4, 12, 36, 68, 100, 1028, 2044])
@pytest.mark.parametrize("res", ["f32", "bf16"])
def test_odd_widths_of_fp32_layers(occ, d, res):
    """fp32 layers take any multiple of 4: rows that are no whole 16 or 32 bytes."""
    for gate in ("channel", "token"):
        c = Case(23, d, "f32", res, gate=gate, seed=d)
        check_forward(occ, c)
        check_backward(occ, c)


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("d", [192, 2048, 5632])
def test_every_combination_of_norms_and_gates(occ, d, post, pre, gate):
    for dtype, res in (("bf16", "bf16"), ("f32", "f32")):
        c = Case(70, d, dtype, res, post, pre, gate, seed=3)
        check_forward(occ, c)
        check_backward(occ, c)


@pytest.mark.parametrize("d", [64, 2048, 16384])
def test_norm_before_the_first_block(occ, d):
    c = Case(45, d, "bf16", "bf16", post=False, y=False)
    check_forward(occ, c)
    check_backward(occ, c)
    check_backward(occ, c, dr_out=False)


@pytest.mark.parametrize("T", [1500, 5000])
def test_many_rows(occ, T):
    """More rows than CTAs: every CTA takes several."""
    c = Case(T, 256, "bf16", "f32", gate="token", seed=9)
    check_forward(occ, c)
    if T <= 1500:
        check_backward(occ, c)


def test_in_place_residual_and_missing_gradient(occ):
    c = Case(200, 2048, "bf16", "bf16", gate="token", seed=4)
    check_forward(occ, c, inplace=True)
    check_backward(occ, c, inplace=True)
    check_backward(occ, c, dr_out=False)


def test_zero_rows_and_rows_of_one_value(occ):
    """A zero block output gives b = 0; a zero stream gives x = 0; no NaN anywhere."""
    c = Case(8, 512, "bf16", "bf16", gate="channel", seed=5)
    c.y[1] = 0
    c.y[2], c.r[2] = 0, 0
    c.r[3] = 0
    c.dr_out[4], c.dx[4] = 0, 0
    c.y[5], c.r[5] = 3.0, -2.0
    check_forward(occ, c)
    check_backward(occ, c)


def test_large_and_small_magnitudes(occ):
    """Rows of 1e15 and 1e-15 side by side (squares up to 1e30 stay finite)."""
    c = Case(6, 256, "f32", "f32", seed=6)
    c.y[0] *= 1e15
    c.y[1] *= 1e-15
    c.r[2] *= 1e15
    for k in ("y", "r"):
        setattr(c, k, rounded(getattr(c, k), "f32"))
    check_forward(occ, c)


def test_no_rows(occ):
    c = Case(0, 128, "bf16", "bf16", gate="channel")
    check_forward(occ, c)
    ds = c.desc(occ)
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(0, 128, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(128, device="cuda")
    o = [torch.full((128,), 7.0, device="cuda") for _ in range(3)]
    occ.occult_block_norm_bwd(ds, c.opt(occ), e, e, e, torch.empty(16, dtype=torch.uint8, device="cuda"),
                              dx=f, y=f, w_post=w, gate=one, w_pre=w, rstd_post=one, rstd_pre=one,
                              dy=e, dw_post=o[0], dgate=o[1], dw_pre=o[2])
    assert not any(t.any() for t in o)


def test_backward_is_bit_reproducible_and_stream_ordered(occ):
    """Two runs on a side stream give the same bits, behind the work queued there."""
    c = Case(700, 2048, "bf16", "bf16", gate="channel", seed=8)
    ds, opt = c.desc(occ), c.opt(occ)
    s = torch.cuda.Stream()
    ins = {k: dev(getattr(c, k), t) for k, t in (("dr_out", c.res), ("dx", "f32"), ("r", c.res),
                                                 ("y", "f32"), ("w_post", c.dtype),
                                                 ("w_pre", c.dtype), ("g", "f32"))}
    rs = torch.rand(c.T, device="cuda") + 0.5
    ws = torch.empty(occ.workspace_size(ds, occ.WS_BLOCK_NORM_BWD), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = []
    for _ in range(2):
        o = [torch.empty(c.T, c.d, dtype=torch.bfloat16, device="cuda") for _ in range(2)] \
            + [torch.empty(c.d, device="cuda") for _ in range(3)]
        late = torch.empty_like(ins["dx"])
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            late.copy_(ins["dx"])
            occ.occult_block_norm_bwd(ds, opt, ins["dr_out"], ins["r"], o[0], ws, dx=late,
                                      y=ins["y"], w_post=ins["w_post"], gate=ins["g"],
                                      w_pre=ins["w_pre"], rstd_post=rs, rstd_pre=rs, dy=o[1],
                                      dw_post=o[2], dgate=o[3], dw_pre=o[4])
        s.synchronize()
        got.append([t.clone() for t in o])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_binding_refuses_strided_and_wrong_types(occ):
    c = Case(4, 128, "bf16", "bf16")
    r = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")[:, :128]
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        occ.occult_block_norm(c.desc(occ), c.opt(occ), r, w_pre=w, x=x)
    with pytest.raises(ValueError):
        occ.occult_block_norm(c.desc(occ), c.opt(occ), x.float(), w_pre=w, x=x)
    with pytest.raises(ValueError):
        occ.occult_block_norm(c.desc(occ), c.opt(occ), x, w_pre=w, x=x[:3].contiguous())
    with pytest.raises(occ.OccultError):      # y without its residual output
        occ.occult_block_norm(c.desc(occ), c.opt(occ), x, y=torch.zeros(4, 128, device="cuda"))


def test_offsets_past_32_bits(occ):
    """2^31 elements and more (T = 1048600, d = 2048): the last rows, both directions."""
    T, d, k = 1048600, 2048, 40
    ds = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, d=d, inter=64))
    opt = occ.occult_norm_t(EPS, 0.75, occ.GATE_TOKEN, occ.OCCULT_BF16)
    c = Case(k, d, "bf16", "bf16", gate="token", seed=12)
    z = lambda dt: torch.zeros(T, d, dtype=dt, device="cuda")  # noqa: E731
    r, y, r_out, x = z(torch.bfloat16), z(torch.float32), z(torch.bfloat16), z(torch.bfloat16)
    gate = torch.ones(T, device="cuda")
    rp, rq = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    r[-k:], y[-k:], gate[-k:] = dev(c.r, "bf16"), dev(c.y, "f32"), dev(c.g, "f32").view(-1)
    w_post, w_pre = dev(c.w_post, "bf16"), dev(c.w_pre, "bf16")
    occ.occult_block_norm(ds, opt, r, y=y, w_post=w_post, gate=gate, w_pre=w_pre, r_out=r_out, x=x,
                          rstd_post=rp, rstd_pre=rq)
    want = onorm.forward(c.r, c.y, c.w_post, c.g, c.w_pre, EPS, 0.75)
    for got, key in ((r_out, "r_out"), (x, "x")):
        a, b = got[-k:].double().cpu().numpy(), want[key]
        assert np.abs(a - b).max() <= 2.0 ** -7 * np.abs(b).max()
        assert not got[:-k:4099].any()
    del x
    dx = z(torch.float32)
    dx[-k:] = dev(c.dx, "f32")
    dr_out = r.zero_()
    dr_out[-k:] = dev(c.dr_out, "bf16")
    dy = z(torch.bfloat16)
    sums = [torch.empty(d, device="cuda") for _ in range(2)]
    ws = torch.empty(occ.workspace_size(ds, occ.WS_BLOCK_NORM_BWD), dtype=torch.uint8, device="cuda")
    saved = r_out[-k:].double().cpu().numpy()
    dgate = torch.empty(T, device="cuda")
    occ.occult_block_norm_bwd(ds, opt, dr_out, r_out, dr_out, ws, dx=dx, y=y, w_post=w_post,
                              gate=gate, w_pre=w_pre, rstd_post=rp, rstd_pre=rq, dy=dy,
                              dw_post=sums[0], dgate=dgate, dw_pre=sums[1])
    want = onorm.backward(c.dr_out, c.dx, saved, c.y, c.w_post, c.g, c.w_pre,
                          rp[-k:].double().cpu().numpy(), rq[-k:].double().cpu().numpy(), 0.75)
    for got, key in ((dr_out[-k:], "dr"), (dy[-k:], "dy"), (sums[0], "dw_post"), (sums[1], "dw_pre")):
        a, b = got.double().cpu().numpy(), want[key]
        assert np.abs(a - b).max() <= 2.0 ** -7 * np.abs(b).max(), key
    assert not dy[:-k:4099].any()


def test_replays_from_a_cuda_graph(occ):
    c = Case(900, 1024, "bf16", "bf16", gate="channel", seed=14)
    ds, opt = c.desc(occ), c.opt(occ)
    t = {k: dev(getattr(c, k), kind) for k, kind in (("r", "bf16"), ("y", "f32"), ("w_post", "bf16"),
                                                     ("w_pre", "bf16"), ("g", "f32"),
                                                     ("dr_out", "bf16"), ("dx", "f32"))}
    o = {k: torch.zeros(900, 1024, dtype=torch.bfloat16, device="cuda") for k in ("r_out", "x", "dr", "dy")}
    f = {k: torch.zeros(n, device="cuda") for k, n in (("rp", 900), ("rq", 900), ("dw_post", 1024),
                                                       ("dgate", 1024), ("dw_pre", 1024))}
    ws = torch.empty(occ.workspace_size(ds, occ.WS_BLOCK_NORM_BWD), dtype=torch.uint8, device="cuda")

    def run():
        occ.occult_block_norm(ds, opt, t["r"], y=t["y"], w_post=t["w_post"], gate=t["g"],
                              w_pre=t["w_pre"], r_out=o["r_out"], x=o["x"], rstd_post=f["rp"],
                              rstd_pre=f["rq"])
        occ.occult_block_norm_bwd(ds, opt, t["dr_out"], o["r_out"], o["dr"], ws, dx=t["dx"], y=t["y"],
                                  w_post=t["w_post"], gate=t["g"], w_pre=t["w_pre"],
                                  rstd_post=f["rp"], rstd_pre=f["rq"], dy=o["dy"],
                                  dw_post=f["dw_post"], dgate=f["dgate"], dw_pre=f["dw_pre"])

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    t["y"].mul_(0.5)
    t["dx"].add_(1.0)
    run()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in {**o, **f}.items()}
    for v in {**o, **f}.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k, v in {**o, **f}.items():
        assert torch.equal(v, want[k]), k


@pytest.mark.parametrize("res", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8256, 12800, 12864, 16384])
def test_wide_rows(occ, d, res):
    """Rows around what a ring of one row holds (12800 columns with an fp32 stream)."""
    for gate, post in (("channel", True), ("token", True), ("none", False)):
        c = Case(170, d, "bf16", res, post=post, gate=gate, seed=d)
        check_forward(occ, c)
        check_backward(occ, c)


@pytest.mark.parametrize("T,d", [(1500, 4), (1500, 36), (700, 128)])
def test_in_place_narrow_rows(occ, T, d):
    """Neighbouring rows share cache lines while copies run ahead of the stores."""
    c = Case(T, d, "f32", "f32", gate="token", seed=d)
    check_forward(occ, c, inplace=True)
    check_backward(occ, c, inplace=True)


@pytest.mark.parametrize("d,dtype,res", [
    (d, dtype, res) for d in (32, 248, 320, 384, 504, 768, 776, 832, 1408, 1536, 1544, 1600, 2112,
                              2304, 2312, 2368, 2816, 2824, 2880, 4096, 6144, 6152, 6208)
    for dtype, res in TYPES if dtype == "f32" or d % 64 == 0])
def test_every_width_of_many_rows(occ, d, dtype, res):
    """Rows enough for a ring of several each, at the ends of the widths that take the
    same number of warps (bf16 layers take multiples of 64)."""
    c = Case(1237, d, dtype, res, gate="token", seed=d)
    check_forward(occ, c, inplace=True)
    check_backward(occ, c, inplace=True)
    c = Case(700, d, dtype, res, pre=False, gate="channel", seed=d + 1)
    check_forward(occ, c)
    check_backward(occ, c)


@pytest.mark.parametrize("d,dtype", [(64, "f32"), (64, "bf16"), (1408, "bf16"), (2048, "bf16"),
                                     (2304, "bf16"), (4096, "f32"), (8256, "f32"), (16384, "f32"),
                                     (36, "f32")])
@pytest.mark.parametrize("kr,ky,kg", [(50, 50, 0), (-50, -50, 0), (57, 0, -40), (0, 50, -40)])
def test_backward_scales_exactly_with_its_rows(occ, d, dtype, kr, ky, kg):
    """r' times 2^kr, y times 2^ky and dx times 2^kg, the row factors with them: every
    product and sum of the definition is then the same but for a power of two, so that
    nothing but the exponents of the gradients may change, to the last bit.  Magnitudes of
    2^50 = 1e15 and more: the cube of a row's factor is no fp32 number there, though the
    gradients (at least 2^-101 times ones of about one, 2^25 above the least normal
    number) are."""
    T = 37
    c = Case(T, d, dtype, "f32" if dtype == "f32" else "bf16", gate="token", seed=d)
    ds, opt = c.desc(occ), c.opt(occ)
    ws = torch.empty(occ.workspace_size(ds, occ.WS_BLOCK_NORM_BWD), dtype=torch.uint8, device="cuda")
    factor = lambda v: dev(rounded(onorm.rstd(v, 0.0), "f32"), "f32")  # noqa: E731
    rq, rp = factor(c.r), factor(c.y)

    def run(kr, ky, kg):
        o = {k: torch.empty(T, d, dtype=DT[c.res if k == "dr" else c.dtype], device="cuda")
             for k in ("dr", "dy")}
        o.update({k: torch.empty(n, device="cuda") for k, n in (("dw_post", d), ("dgate", T),
                                                                ("dw_pre", d))})
        occ.occult_block_norm_bwd(
            ds, opt, None, dev(c.r * 2.0 ** kr, c.res), o["dr"], ws, dx=dev(c.dx * 2.0 ** kg, "f32"),
            y=dev(c.y * 2.0 ** ky, "f32"), w_post=dev(c.w_post, c.dtype), gate=dev(c.g, "f32"),
            w_pre=dev(c.w_pre, c.dtype), rstd_post=rp * 2.0 ** -ky, rstd_pre=rq * 2.0 ** -kr,
            dy=o["dy"], dw_post=o["dw_post"], dgate=o["dgate"], dw_pre=o["dw_pre"])
        torch.cuda.synchronize()
        return {k: t.double() for k, t in o.items()}

    base, got = run(0, 0, 0), run(kr, ky, kg)
    D = kg - kr                    # of D; dy has y's factor besides, dw_pre only that of dx
    for k, e in (("dr", D), ("dy", D - ky), ("dw_post", D), ("dgate", D), ("dw_pre", kg)):
        want = base[k] * 2.0 ** e
        assert want.isfinite().all() and torch.equal(got[k], want), \
            (k, float((got[k] - want).abs().max() / want.abs().max()))


@pytest.mark.parametrize("d", [64, 2048, 2304, 4096, 16384])
@pytest.mark.parametrize("eps,both", [(1e-26, True), (1e-30, True), (1e-40, False)])
def test_backward_of_zero_rows_at_a_small_eps(occ, d, eps, both, monkeypatch):
    """A zero row has the factor eps^(-1/2), and finite gradients: the means over it are 0.
    (Where both norms see zeros dy has both factors: 1e40 at the least eps.)"""
    monkeypatch.setitem(globals(), "EPS", eps)
    for gate in ("token", "channel"):
        c = Case(20, d, "f32", "f32", gate=gate, seed=15)
        c.y[7] = 0
        if both:
            c.y[3], c.r[3] = 0, 0
        check_backward(occ, c)
