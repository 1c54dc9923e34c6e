"""GPU parity of occult_adamw with the fp64 oracle.

With u = 2^-24 the moments are two rounded products and a sum of them (coefficients
rounded as well): within 4 u of the sum of magnitudes.  The root and the quotient
add 2 + 2 units, so the update is within 24 u of its magnitude plus what the moments'
errors do to it, the parameter within 3 u more.  8-bit codes equal the oracle's
except where the fp64 value in units plus its draw lies within SLACK of a whole
number (the fp32 value is within 8 u of it, up to 32 units of a code: 2^-16), and
then they are neighbours.
"""
import numpy as np
import pytest
import torch

from oracle import adamw as oadam

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SLACK = 2.0 ** -15
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
KINDS = ["f32", "master", "bf16"]


@pytest.fixture(scope="module")
def occ():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_top_route_gb300 import build
    build.build()
    import combine_top_route_gb300 as occ
    occ.lib()
    return occ


def fresh(n, kind, bits, seed, scale=1e-2):
    """One tensor's state on the host (fp64 values that its types hold)."""
    rng = np.random.default_rng(seed)
    f = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731
    s = dict(n=n, kind=kind, bits=bits, first=seed * 1000)
    s["grad"] = f(rng.normal(size=n) * scale)
    w = f(rng.normal(size=n) * 0.05)
    s["master"] = w if kind == "master" else None
    s["param"] = w if kind == "f32" else torch.as_tensor(w).to(torch.bfloat16).double().numpy()
    m, v = rng.normal(size=n) * scale / 3, (rng.normal(size=n) * scale) ** 2
    if bits == 32:
        s["m"], s["v"] = f(m), f(v)
    else:
        half = np.full(n, 0.5)
        s["m"], s["m_exp"], _ = oadam.encode(m, half, 3)
        s["v"], s["v_exp"], _ = oadam.encode(np.sqrt(v), half, 4)
    return s


def upload(s):
    guard = 16
    dt = {"param": torch.float32 if s["kind"] == "f32" else torch.bfloat16, "master": torch.float32,
          "grad": torch.float32}
    st = torch.float32 if s["bits"] == 32 else torch.uint8
    dt.update(m=st, v=st, m_exp=torch.uint8, v_exp=torch.uint8)
    full, view = {}, {}
    for k, t in dt.items():
        if s.get(k) is None:
            full[k] = view[k] = None
            continue
        n = len(s[k])
        full[k] = torch.full((n + guard,), 9, dtype=t, device="cuda")
        full[k][:n] = torch.as_tensor(np.asarray(s[k])).to(t)
        view[k] = full[k][:n]
    view["first"] = s["first"]
    return full, view


def check(occ, s, full, view, t, gs=1.0, seed=5, hyper=HYPER):
    n = s["n"]
    for k, b in full.items():
        if b is not None:
            assert (b[len(s[k]):] == 9).all(), f"{k}: written past its end"
    host = {k: v.double().cpu().numpy() for k, v in view.items() if isinstance(v, torch.Tensor)}
    assert (host["grad"] == s["grad"]).all()
    small = s["bits"] == 8
    m0 = oadam.decode(s["m"], s["m_exp"], 3) if small else s["m"]
    r0 = oadam.decode(s["v"], s["v_exp"], 4) if small else None
    v0 = r0 ** 2 if small else s["v"]
    w0 = s["master"] if s["kind"] == "master" else s["param"]
    w, m, v = oadam.step(w0, s["grad"], m0, v0, t, grad_scale=gs, **hyper)
    g = gs * s["grad"]
    d_m, d_v, d_p = oadam.draws(n, s["first"], seed, t)
    e_m = 4 * U * (np.abs(hyper["beta1"] * m0) + np.abs((1 - hyper["beta1"]) * g)) + 1e-43
    e_v = 6 * U * v + 1e-43
    if not small:
        assert (np.abs(host["m"] - m) <= e_m).all()
        assert (np.abs(host["v"] - v) <= e_v).all()
    else:
        for key, x, d, mant in (("m", m, d_m, 3), ("v", np.sqrt(v), d_v, 4)):
            code, exp, slack = oadam.encode(x, d, mant)
            got_e = host[key + "_exp"].astype(int)
            # the block's exponent: equal unless its largest value is that near a binade
            near = np.abs(got_e - exp)
            assert near.max(initial=0) <= 1 and (near > 0).mean() <= 0.01
            same = np.repeat(near == 0, oadam.BLOCK)[:n]
            got = host[key].astype(int)
            off = (got != code) & same
            a, b = oadam.decode(got, got_e, mant), oadam.decode(code, exp, mant)
            unit = np.exp2(np.frexp(np.maximum(np.abs(a), np.abs(b)))[1] - 1 - mant)
            assert (slack[off] <= SLACK).all(), (key, slack[off].max())
            assert (np.abs(a - b)[off] <= unit[off]).all()
            lib = torch.empty(n, dtype=torch.bfloat16, device="cuda")
            occ.occult_adamw_read(view[key], view[key + "_exp"],
                                  occ.STATE_M if key == "m" else occ.STATE_V, lib)
            assert (lib.double().cpu().numpy() == a).all()
    root = np.sqrt(v / (1 - hyper["beta2"] ** t)) + hyper["eps"]
    upd = hyper["lr"] / (1 - hyper["beta1"] ** t) * m / root
    e_w = 24 * U * np.abs(upd) + np.abs(hyper["lr"] / (1 - hyper["beta1"] ** t) / root) * e_m \
        + 3 * U * np.abs(w0) + 3 * U * np.abs(w) + 1e-43
    if s["kind"] == "f32":
        assert (np.abs(host["param"] - w) <= e_w).all()
    elif s["kind"] == "master":
        assert (np.abs(host["master"] - w) <= e_w).all()
        want = torch.as_tensor(host["master"]).float().to(torch.bfloat16).double().numpy()
        assert (host["param"] == want).all()
    else:
        # one of the two neighbours, the one the draw says unless it is a near tie
        unit = np.exp2(np.frexp(w)[1] - 8.0)
        real = np.abs(w) / unit + d_p
        want = np.sign(w) * np.floor(real) * unit
        off = np.abs(host["param"] - want) > 1e-43
        tie = np.abs(real - np.rint(real)) <= e_w / unit + 2.0 ** -20
        assert tie[off].all()
        assert (np.abs(host["param"] - w) <= unit * 1.001 + e_w).all()


def step(occ, views, t, bits, gs=None, seed=5, hyper=HYPER, stream=None):
    opt = occ.occult_adamw_t(step=t, state_bits=bits, seed=seed,
                             grad_scale=None if gs is None else gs.data_ptr(), **hyper)
    occ.occult_adamw(opt, occ.adamw_table(views), stream)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [1, 3, 4, 127, 255, 256, 257, 2047, 8192, 8193, 70001])
def test_one_tensor(occ, n, bits, kind):
    s = fresh(n, kind, bits, seed=n % 97)
    full, view = upload(s)
    gs = torch.full((1,), 0.625, device="cuda")
    step(occ, [view], 3, bits, gs)
    check(occ, s, full, view, 3, gs=0.625)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [2, 40, 256, 300])
def test_many_tensors_of_all_kinds(occ, bits, count):
    """More tensors than one launch takes, empty ones among them."""
    rng = np.random.default_rng(count)
    sizes = [int(x) for x in np.exp(rng.uniform(0, 9, count))]
    sizes[count // 2] = 0
    all_s = [fresh(n, KINDS[i % 3], bits, seed=i) for i, n in enumerate(sizes)]
    up = [upload(s) for s in all_s]
    step(occ, [v for _, v in up], 10, bits)
    for s, (full, view) in zip(all_s, up):
        if s["n"]:
            check(occ, s, full, view, 10)


@pytest.mark.parametrize("kind", KINDS)
def test_fresh_8bit_state_first_step(occ, kind):
    """All-zero codes and exponents; some gradients zero."""
    s = fresh(5000, kind, 8, seed=1)
    for k in ("m", "v", "m_exp", "v_exp"):
        s[k][:] = 0
    s["grad"][::3] = 0
    s["grad"][256:512] = 0
    full, view = upload(s)
    step(occ, [view], 1, 8)
    check(occ, s, full, view, 1)
    assert not view["m"][256:512].any() and not view["v"][256:512].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_cut_tensors_give_the_same_bits(occ, bits):
    """A tensor cut at whole state blocks, with `first` moved along, steps the same."""
    s = fresh(4096, "bf16", bits, seed=2)
    _, a = upload(s)
    _, b = upload(s)
    step(occ, [a], 4, bits)
    cuts = [0, 256, 1536, 4096]
    parts = []
    for lo, hi in zip(cuts, cuts[1:]):
        p = {k: b[k][lo:hi] for k in ("param", "grad", "m", "v")}
        p["first"] = b["first"] + lo
        if bits == 8:
            p.update({k: b[k][lo // 256:hi // 256] for k in ("m_exp", "v_exp")})
        parts.append(p)
    step(occ, parts, 4, bits)
    for k in ("param", "m", "v"):
        assert torch.equal(a[k], b[k])


@pytest.mark.parametrize("kind", KINDS)
def test_infinite_gradients_stay_in_their_block(occ, kind):
    s = fresh(1024, kind, 8, seed=3)
    s["grad"][300] = np.inf
    s["grad"][700] = np.nan
    _, view = upload(s)
    step(occ, [view], 2, 8)
    vals = torch.empty(1024, dtype=torch.bfloat16, device="cuda")
    for key, which in (("m", occ.STATE_M), ("v", occ.STATE_V)):
        occ.occult_adamw_read(view[key], view[key + "_exp"], which, vals)
        nan = vals.isnan().cpu().numpy().reshape(4, 256).all(axis=1)
        assert nan.tolist() == [False, True, True, False]
    p = view["param"].float().cpu().numpy()
    bad = ~np.isfinite(p)
    assert bad[[300, 700]].all() and bad.sum() == 2
    step(occ, [view], 3, 8)      # from then on the block is NaN
    bad = ~np.isfinite(view["param"].float().cpu().numpy())
    assert bad[256:768].all() and not bad[:256].any() and not bad[768:].any()


def test_extreme_magnitudes(occ):
    """Gradients from 1e-30 to 1e15 in one block; denormal and zero ones."""
    for kind in KINDS:
        s = fresh(512, kind, 8, seed=4)
        s["grad"][:256] = (np.sign(s["grad"][:256])
                           * 10.0 ** np.linspace(-30, 15, 256)).astype(np.float32)
        s["grad"][256:300] = 0
        s["grad"][300] = float(np.float32(1e-42))
        full, view = upload(s)
        step(occ, [view], 2, 8)
        check(occ, s, full, view, 2)


def test_rounding_by_draw_keeps_small_updates(occ):
    """A bf16 parameter of 1 with updates of 1/64 unit, 512 steps: on average they
    arrive (rounding to nearest would lose all of them)."""
    n, steps = 4096, 512
    unit = 2.0 ** -8                       # spacing below 1
    lr = unit / 64
    view = dict(param=torch.ones(n, dtype=torch.bfloat16, device="cuda"),
                grad=torch.ones(n, device="cuda"), m=torch.zeros(n, device="cuda"),
                v=torch.zeros(n, device="cuda"))
    for t in range(1, steps + 1):
        opt = occ.occult_adamw_t(lr=lr, beta1=0.9, beta2=0.95, eps=1e-12, weight_decay=0.0, step=t,
                                 state_bits=32, seed=11)
        occ.occult_adamw(opt, occ.adamw_table([view]))
    mean = float(view["param"].double().mean())
    # each step adds a variance of at most unit^2 / 64 an element
    assert abs((1 - mean) - steps * lr) < 6 * unit * np.sqrt(steps / 64 / n) + 1e-3 * steps * lr


def test_8bit_states_track_32bit_ones(occ):
    """400 steps of noisy gradients: the parameters with 8-bit states stay within a
    few per cent of the distance that 32-bit states take them."""
    n = 1 << 14
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randn(n, generator=g, device="cuda") * 0.02
    drift = torch.randn(n, generator=g, device="cuda") * 1e-3
    sides = []
    for bits in (32, 8):
        st = torch.float32 if bits == 32 else torch.uint8
        t = dict(param=w.clone(), grad=torch.empty(n, device="cuda"),
                 m=torch.zeros(n, dtype=st, device="cuda"), v=torch.zeros(n, dtype=st, device="cuda"))
        if bits == 8:
            t.update(m_exp=torch.zeros(n // 256, dtype=torch.uint8, device="cuda"),
                     v_exp=torch.zeros(n // 256, dtype=torch.uint8, device="cuda"))
        sides.append(t)
    for i in range(1, 401):
        grad = drift + 1e-3 * torch.randn(n, generator=g, device="cuda")
        for bits, t in zip((32, 8), sides):
            t["grad"].copy_(grad)
            opt = occ.occult_adamw_t(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0,
                                     step=i, state_bits=bits, seed=3)
            occ.occult_adamw(opt, occ.adamw_table([t]))
    a, b = (t["param"].double() for t in sides)
    moved = float((a - w).norm())
    assert float((a - b).norm()) < 0.1 * moved
    assert abs(float(((b - w) * (a - w)).sum()) / moved ** 2 - 1) < 0.02


def test_on_a_side_stream_and_in_a_graph(occ):
    s = fresh(3000, "master", 8, seed=6)
    _, a = upload(s)
    _, b = upload(s)
    step(occ, [a], 7, 8)
    st = torch.cuda.Stream()
    table = occ.adamw_table([b])
    opt = occ.occult_adamw_t(step=7, state_bits=8, seed=5, **HYPER)
    keep = {k: b[k].clone() for k in ("param", "master", "m", "v", "m_exp", "v_exp")}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        occ.occult_adamw(opt, table)
    for k, t in keep.items():
        assert torch.equal(t, b[k])
    g.replay()
    torch.cuda.synchronize()
    for k in keep:
        assert torch.equal(a[k], b[k])


def test_offsets_past_32_bits(occ):
    """A tensor of more than 2^31 elements (bf16, 8-bit states: 17 GB): its last blocks."""
    n = (1 << 31) + 777
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    me, ve = (torch.zeros(-(-n // 256), dtype=torch.uint8, device="cuda") for _ in range(2))
    tail = 1024 + 9
    lo = n - tail
    lo -= lo % 256
    rng = np.random.default_rng(1)
    tg = (rng.normal(size=n - lo) * 1e-2).astype(np.float32)
    tp = torch.as_tensor(rng.normal(size=n - lo) * 0.05).to(torch.bfloat16)
    g[lo:] = torch.as_tensor(tg).cuda()
    p[lo:] = tp.cuda()
    step(occ, [dict(param=p, grad=g, m=m, v=v, m_exp=me, v_exp=ve, first=0)], 1, 8)
    k = n - lo
    s = dict(n=k, kind="bf16", bits=8, first=lo, grad=tg.astype(np.float64),
             param=tp.double().numpy(), master=None, m=np.zeros(k, int), v=np.zeros(k, int),
             m_exp=np.zeros(-(-k // 256), int), v_exp=np.zeros(-(-k // 256), int))
    view = dict(param=p[lo:], grad=g[lo:], m=m[lo:], v=v[lo:], m_exp=me[lo // 256:],
                v_exp=ve[lo // 256:])
    check(occ, s, {}, view, 1)
    assert not p[:lo:4096].any() and not m[:lo:4096].any()


@pytest.mark.parametrize("large", KINDS)
@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_steps_the_same_beside_others(occ, bits, large):
    """One kind large enough for launches of its own, the others small: the bits that
    each tensor gets when it is stepped alone."""
    big = (1 << 25) + 300
    st = torch.float32 if bits == 32 else torch.uint8
    gen = torch.Generator(device="cuda").manual_seed(12)

    def tensor(kind, n, first):
        w = torch.randn(n, generator=gen, device="cuda") * 0.05
        t = dict(param=w if kind == "f32" else w.to(torch.bfloat16), first=first,
                 grad=torch.randn(n, generator=gen, device="cuda") * 1e-2,
                 m=torch.zeros(n, dtype=st, device="cuda"), v=torch.zeros(n, dtype=st, device="cuda"))
        if kind == "master":
            t["master"] = w
        if bits == 8:
            t.update({k: torch.zeros(-(-n // 256), dtype=torch.uint8, device="cuda")
                      for k in ("m_exp", "v_exp")})
        return t

    together = [tensor(kind, big if kind == large and i == 1 else 1000 + 7 * i, 1000 * i)
                for i in range(3) for kind in KINDS]
    alone = [{k: x.clone() if isinstance(x, torch.Tensor) else x for k, x in t.items()}
             for t in together]
    for t in (1, 2):
        step(occ, together, t, bits)
        for x in alone:
            step(occ, [x], t, bits)
    for a, b in zip(together, alone):
        for k in a:
            assert torch.equal(a[k], b[k]) if isinstance(a[k], torch.Tensor) else a[k] == b[k], k


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("many", [1, 150, 256])
def test_every_cta_finds_its_tensor(occ, bits, many):
    """Tensors of a block next to ones of thousands, in every order: a launch of more
    CTAs than its search has spans, against each tensor alone."""
    sizes = [1 + 300 * (i % 5) for i in range(many)] + [5000000]
    for order in (sizes, sizes[::-1], sizes[::2] + sizes[1::2][::-1]):
        order = order[-256:]
        gen = torch.Generator(device="cuda").manual_seed(many)
        st = torch.float32 if bits == 32 else torch.uint8
        together = []
        for i, n in enumerate(order):
            t = dict(param=torch.randn(n, generator=gen, device="cuda").to(torch.bfloat16),
                     grad=torch.randn(n, generator=gen, device="cuda"), first=i * 7,
                     m=torch.zeros(n, dtype=st, device="cuda"),
                     v=torch.zeros(n, dtype=st, device="cuda"))
            if bits == 8:
                t.update({k: torch.zeros(-(-n // 256), dtype=torch.uint8, device="cuda")
                          for k in ("m_exp", "v_exp")})
            together.append(t)
        alone = [{k: x.clone() if isinstance(x, torch.Tensor) else x for k, x in t.items()}
                 for t in together]
        step(occ, together, 1, bits)
        for x in alone:
            step(occ, [x], 1, bits)
        for a, b in zip(together, alone):
            assert all(torch.equal(a[k], b[k]) for k in a if k != "first")
