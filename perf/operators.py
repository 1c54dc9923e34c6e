"""Workloads of the operators around the MoE layer in a training step.

Three operators and their cases: the block norm (RMSNorm before and after a
block with its gate and residual scale, forward and backward), the router's
balance loss with its gradient, and the AdamW step over many tensors.  ``run``
makes one call of an operator: in its plain form (elementary torch operations in
fp32) or, with ``own`` set, through ``combine_top_route_gb300``.
"""
import itertools
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32

# AdamW hyperparameters (those MoE language models are commonly trained with)
LR, BETA1, BETA2, EPS, DECAY = 4e-4, 0.9, 0.95, 1e-8, 0.1
STATE_BLOCK = 256
# multipliers of the rounding draw (fractional parts of sqrt 3 and sqrt 5, odd)
MUL1, MUL2, M32 = 0xBB67AE85, 0x3C6EF373, 0xFFFFFFFF


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token: the norm after a block, its residual sum and the next
        # block's norm at the layer width; latency is all that counts
        norm("norm_one_token", False, 1, 2048, "bf16", "bf16", True, True, "channel"),
        # 512 concurrent decode tokens of a pre-norm model: residual sum and norm
        norm("norm_decode_512", False, 512, 2048, "bf16", "bf16", False, True, "none"),
        # the training step's 32768 tokens, norms on both sides, channel gates
        norm("norm_train", False, 32768, 2048, "bf16", "bf16", True, True, "channel"),
        # the small fp32 layer with a ragged batch and a gate for every token
        norm("norm_grad_f32_small", True, 257, 64, "f32", "f32", True, True, "token"),
        # the training step's backward, norms on both sides, channel gates
        norm("norm_grad_train", True, 32768, 2048, "bf16", "bf16", True, True, "channel"),
        # backward at prefill length with an fp32 residual stream, token gates
        norm("norm_grad_f32_stream", True, 16383, 2048, "bf16", "f32", True, True, "token"),
        # router of the small layer: 256 tokens, one group
        balance("balance_small", 256, 8, 2, 4, 0, False),
        # router of the training step, one group over the whole batch
        balance("balance_train", 32768, 64, 8, 16, 0, False),
        # sequence-wise balance of 32 padded sequences over 256 experts
        balance("balance_sequences", 131072, 256, 8, 32, 4096, True),
        # norms, gates and biases of a model: many small fp32 tensors, odd sizes
        adamw("adamw_many_small", 200, 1 << 19, "f32", 32),
        # one layer's experts and router (w1, w2, router): bf16 with fp32 masters
        adamw("adamw_layer", 3, 402784256, "bf16_master", 32),
        # the same layer with 8-bit states and no master copy
        adamw("adamw_layer_8bit", 3, 402784256, "bf16", 8),
    ]


def norm(name, grad, T, d, dtype, res, post, pre, gate):
    return {"name": name, "op": "norm_grad" if grad else "norm", "T": T, "d": d, "dtype": dtype,
            "res": res, "post": post, "pre": pre, "gate": gate}


def balance(name, T, n_experts, top_k, n_vdev, group_len, masked):
    return {"name": name, "op": "balance", "T": T, "n_experts": n_experts, "top_k": top_k,
            "n_vdev": n_vdev, "group_len": group_len, "masked": masked}


def adamw(name, tensors, total, kind, bits):
    return {"name": name, "op": "adamw", "tensors": tensors, "total": total, "kind": kind,
            "bits": bits}


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "balance", "adamw"])
    if op in ("norm", "norm_grad"):
        d = rng.choice([64, 192, 320, 512, 768, 1024, 1408, 2048, 2112, 2816, 4096, 5632])
        T = log_int(rng, 1, 32768 * 2048 // max(d, 2048))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        c = norm("", op == "norm_grad", T + (T == 3072), d, dtype,
                 rng.choice(["bf16", "f32"]) if dtype == "bf16" else "f32", post, pre,
                 rng.choice(["none", "channel", "token"]))
    elif op == "balance":
        n_vdev = rng.choice([1, 2, 4, 8, 16])
        n_experts = n_vdev * rng.randint(max(1, 4 // n_vdev), 256 // n_vdev)
        T = log_int(rng, 16, 131072)
        c = balance("", T + (T == 3072), n_experts, rng.randint(1, min(16, n_experts)), n_vdev,
                    rng.choice([0, 0, max(1, T // rng.randint(2, 24))]), rng.random() < 0.5)
    else:
        total = log_int(rng, 4096, 300_000_000)
        c = adamw("", rng.randint(1, 200), total, rng.choice(["f32", "bf16_master", "bf16"]),
                  rng.choice([8, 32]))
    del c["name"]
    return c


def sizes_of(case):
    """Elements of every tensor: weights of the layer for three, else uneven odd sizes."""
    n, total = case["tensors"], case["total"]
    if n == 3 and total == 402784256:
        return [64 * 2 * 1024 * 2048, 64 * 2048 * 1024, 64 * 2048]
    w = np.random.RandomState(n).lognormal(0.0, 1.5, n)
    return [max(1, int(total * x)) for x in w / w.sum()]


def starts_of(sizes):
    """Offsets of the tensors in their flat bucket: whole state blocks apart."""
    return list(itertools.accumulate([0] + [-(-n // STATE_BLOCK) * STATE_BLOCK for n in sizes]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(case, seed):
    return {"norm": prepare_norm, "norm_grad": prepare_norm, "balance": prepare_balance,
            "adamw": prepare_adamw}[case["op"]](case, seed)


def prepare_norm(case, seed):
    g = generator(seed)
    T, d = case["T"], case["d"]
    dt, rt = (BF16 if case[k] == "bf16" else F32 for k in ("dtype", "res"))
    s = dict(case, eps=1e-6, res_scale=1.0 if case["gate"] == "none" else 0.9)
    # a residual stream a few times as large as the block outputs added to it
    s["r"] = (2.5 * torch.randn(T, d, generator=g, device=DEV)).to(rt)
    s["y"] = 0.7 * torch.randn(T, d, generator=g, device=DEV)
    s["w_post"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt) if case["post"] else None
    s["w_pre"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt) if case["pre"] else None
    n = {"none": 0, "channel": d, "token": T}[case["gate"]]
    s["gate_v"] = 0.5 + 0.3 * torch.randn(n, generator=g, device=DEV) if n else None
    rows = lambda dtype: torch.empty(T, d, dtype=dtype, device=DEV)  # noqa: E731
    if case["op"] == "norm":
        s.update(r_out=rows(rt), x=rows(dt) if case["pre"] else None,
                 rstd_post=torch.empty(T, device=DEV) if case["post"] else None,
                 rstd_pre=torch.empty(T, device=DEV) if case["pre"] else None)
        return s
    # the backward's inputs: what the forward saved, and the gradients that arrive
    s["rstd_post"] = (s["y"].square().mean(1) + s["eps"]).rsqrt() if case["post"] else None
    s["r_out"] = s.pop("r")
    s["rstd_pre"] = (s["r_out"].float().square().mean(1) + s["eps"]).rsqrt() if case["pre"] else None
    s["dr_out"] = torch.randn(T, d, generator=g, device=DEV).to(rt)
    s["dx"] = torch.randn(T, d, generator=g, device=DEV) if case["pre"] else None
    s.update(dr=rows(rt), dy=rows(dt),
             dw_post=torch.empty(d, device=DEV) if case["post"] else None,
             dgate=torch.empty(n, device=DEV) if n else None,
             dw_pre=torch.empty(d, device=DEV) if case["pre"] else None)
    return s


def prepare_balance(case, seed):
    g = generator(seed)
    T, E, k = case["T"], case["n_experts"], case["top_k"]
    s = dict(case, coef=0.01, coef_dev=0.005, coef_z=0.001)
    s["L"] = case["group_len"] or T
    s["G"] = -(-T // s["L"])
    boost = torch.rand(16, E, generator=g, device=DEV) < 10 / 64
    cluster = torch.randint(0, 16, (T,), generator=g, device=DEV)
    z = torch.randn(T, E, generator=g, device=DEV) + 3.0 * boost[cluster]
    s["ids"] = z.topk(k, dim=1).indices.to(torch.int32).contiguous()
    s["mask"] = None
    if case["masked"]:
        # sequences padded at their ends, the last group (if it is not all) empty;
        # what the padding's rows hold is not a number
        pos = torch.arange(T, device=DEV)
        keep = torch.rand(s["G"], generator=g, device=DEV) * 0.5 + 0.5
        keep = torch.where((torch.arange(s["G"], device=DEV) == s["G"] - 1) & (s["G"] > 1), 0.0, keep)
        s["mask"] = (pos % s["L"] < (keep * s["L"]).ceil()[pos // s["L"]]).to(torch.uint8)
        z = torch.where(s["mask"][:, None] != 0, z, float("nan"))
    s["logits"] = z.contiguous()
    s["e2v"] = (torch.randperm(E, generator=g, device=DEV) % case["n_vdev"]).to(torch.int32)
    # the gradient that came through the gates, which the balance gradient adds to
    s["dlogits"] = 1e-4 * torch.randn(T, E, generator=g, device=DEV)
    s["dloss"] = torch.full((1,), 1.0, device=DEV)
    s["counts"] = torch.empty(s["G"], E, dtype=torch.int32, device=DEV)
    s["grad_w"] = torch.empty(s["G"] * E + 1, device=DEV)
    s["loss"] = torch.empty(4, device=DEV)
    return s


def prepare_adamw(case, seed):
    g = generator(seed)
    sizes = sizes_of(case)
    starts = starts_of(sizes)
    n = starts[-1]
    live = torch.zeros(n, dtype=torch.bool, device=DEV)
    [live[a:a + m].fill_(True) for a, m in zip(starts, sizes)]
    rnd = lambda std: torch.randn(n, generator=g, device=DEV).mul_(std).mul_(live)  # noqa: E731
    s = dict(case, sizes=sizes, starts=starts, n=n, step=100, seed=seed & 0x7FFFFFFF)
    w = rnd(0.02)
    s["master"] = w if case["kind"] == "bf16_master" else None
    s["param"] = w if case["kind"] == "f32" else w.to(BF16)
    s["grad"] = rnd(1e-3)
    s["grad_scale"] = torch.full((1,), 0.8, device=DEV)
    m, v = rnd(4e-4), rnd(1e-3).square_()
    if case["bits"] == 32:
        s.update(m=m, v=v, m_exp=None, v_exp=None)
    else:
        half = torch.full((n,), 0x8000, dtype=torch.int32, device=DEV)
        s["m"], s["m_exp"] = pack8(m, half, 3)
        s["v"], s["v_exp"] = pack8(v.sqrt_(), half, 4)
    s["m_val"] = torch.empty(n, dtype=BF16, device=DEV) if case["bits"] == 8 else None
    s["v_val"] = torch.empty(n, dtype=BF16, device=DEV) if case["bits"] == 8 else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return {"norm": own_norm, "norm_grad": own_norm_grad, "balance": own_balance,
                "adamw": own_adamw}[state["op"]](state)
    return {"norm": plain_norm, "norm_grad": plain_norm_grad, "balance": plain_balance,
            "adamw": plain_adamw}[state["op"]](state)


def gate_of(s):
    """The gate as something that multiplies [T, d] rows."""
    return 1.0 if s["gate"] == "none" else s["gate_v"] if s["gate"] == "channel" else s["gate_v"][:, None]


def plain_norm(s):
    out = {}
    b = s["y"]
    if s["post"]:
        out["rstd_post"] = ((b * b).mean(1) + s["eps"]).rsqrt()
        b = b * out["rstd_post"][:, None] * s["w_post"].float()
    r = s["res_scale"] * s["r"].float() + gate_of(s) * b
    out["r_out"] = r.to(s["r"].dtype)
    if s["pre"]:
        out["rstd_pre"] = ((r * r).mean(1) + s["eps"]).rsqrt()
        out["x"] = (r * out["rstd_pre"][:, None] * s["w_pre"].float()).to(s["w_pre"].dtype)
    return out


def plain_norm_grad(s):
    out = {}
    D = s["dr_out"].float()
    if s["pre"]:
        xhat = s["r_out"].float() * s["rstd_pre"][:, None]
        g = s["dx"] * s["w_pre"].float()
        D = D + s["rstd_pre"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
        out["dw_pre"] = (s["dx"] * xhat).sum(0)
    out["dr"] = (s["res_scale"] * D).to(s["dr_out"].dtype)
    yhat = s["y"] * s["rstd_post"][:, None] if s["post"] else s["y"]
    branch = yhat * s["w_post"].float() if s["post"] else yhat
    if s["gate"] != "none":
        out["dgate"] = (D * branch).sum(0 if s["gate"] == "channel" else 1)
    u = gate_of(s) * D
    if s["post"]:
        out["dw_post"] = (u * yhat).sum(0)
        u = u * s["w_post"].float()
        u = s["rstd_post"][:, None] * (u - yhat * (u * yhat).mean(1, keepdim=True))
    out["dy"] = u.to(BF16 if s["dtype"] == "bf16" else F32)
    return out


def grouped(s, v):
    """Rows [T, ...] as groups [G, L, ...], the last one filled up with zeros."""
    pad = s["G"] * s["L"] - s["T"]
    if pad:
        v = torch.cat([v, v.new_zeros((pad,) + tuple(v.shape[1:]))])
    return v.view((s["G"], s["L"]) + tuple(v.shape[1:]))


def plain_balance(s):
    T, E, k, G, L = s["T"], s["n_experts"], s["top_k"], s["G"], s["L"]
    on = torch.ones(T, device=DEV) if s["mask"] is None else (s["mask"] != 0).float()
    z = torch.where(on[:, None] > 0, s["logits"], 0.0)
    top = z.amax(1, keepdim=True)
    e = (z - top).exp()
    Z = e.sum(1, keepdim=True)
    p = e / Z * on[:, None]
    lse = (top + Z.log())[:, 0] * on
    # tokens of a group, slots and probability of each expert in it
    N = grouped(s, on).sum(1)
    group = torch.arange(T, device=DEV) // L
    where = (group[:, None] * E + s["ids"]).view(-1)
    ones = on.to(torch.int32)[:, None].expand(T, k).reshape(-1)
    counts = torch.zeros(G * E, dtype=torch.int32, device=DEV).scatter_add_(0, where, ones).view(G, E)
    share = grouped(s, p).sum(1) / N.clamp(min=1)[:, None]
    groups, tokens = (N > 0).sum().clamp(min=1), N.sum().clamp(min=1)
    f = counts * (E / k) / N.clamp(min=1)[:, None]
    member = (s["e2v"][:, None] == torch.arange(s["n_vdev"], device=DEV)).float()
    f_dev = (f @ member) / member.sum(0).clamp(min=1)
    bal = (f * share).sum() / groups
    dev = (f_dev * (share @ member)).sum() / groups
    sq = (lse * lse).sum() / tokens
    loss = torch.stack([s["coef"] * bal + s["coef_dev"] * dev + s["coef_z"] * sq, bal, dev, sq])
    # dz = p (w - sum p w) + 2 cz / N lse p
    w = (s["coef"] * f + s["coef_dev"] * (f_dev @ member.T)) / (groups * N.clamp(min=1))[:, None]
    w = w[group]
    dz = p * (w - (p * w).sum(1, keepdim=True)) + (2 * s["coef_z"] / tokens) * lse[:, None] * p
    s["dlogits"].add_(s["dloss"] * dz)
    return {"loss": loss, "counts": counts, "dlogits": s["dlogits"]}


def mix(x):
    """A 32-bit hash of x (int64 tensor or int in [0, 2^32))."""
    x = (x * MUL1) & M32
    x = x ^ (x >> 15)
    x = (x * MUL2) & M32
    return x ^ (x >> 16)


def draws(n, seed, step):
    """Three 16-bit draws for each of n positions: of m, of sqrt(v), of the parameter."""
    key = mix((seed + mix(step & M32)) & M32)
    h = mix((torch.arange(n, device=DEV) + key) & M32)
    return (h & 0xFFFF).int(), (h >> 16).int(), (((h * MUL1) & M32) >> 16).int()


def pack8(x, dither, mant):
    """Codes and block exponents of fp32 x: `mant` mantissa bits, 4 exponent bits
    under the block's largest exponent, a sign where that leaves room."""
    cut = 23 - mant
    bits = x.view(torch.int32) & 0x7FFFFFFF
    top = bits.view(-1, STATE_BLOCK).amax(1)
    exp = ((top + ((1 << cut) - 1)) >> 23).clamp(min=16)
    exp = torch.where(top >= 0x7F800000, 255, exp)
    low = ((exp - 15) << mant).repeat_interleave(STATE_BLOCK)
    k = ((bits + (dither << (cut - 16))) >> cut) - low
    k = k.clamp(min=0, max=(16 << mant) - 1)
    if mant == 3:
        k = torch.where((x < 0) & (k > 0), k + 128, k)
    else:
        k = torch.where((x > 0) & (k == 0), 1, k)
    return k.to(torch.uint8), exp.to(torch.uint8)


def unpack8(code, exp, mant):
    """The fp32 values that pack8's codes stand for."""
    e = exp.int().repeat_interleave(STATE_BLOCK)
    mag = code.int() & ((16 << mant) - 1)
    x = ((mag + ((e - 15) << mant)) << (23 - mant)).view(F32)
    x = torch.where(mag == 0, 0.0, x)
    x = torch.where(e == 255, float("nan"), x)
    return torch.where(code >= 128, -x, x) if mant == 3 else x


def plain_adamw(s):
    s["step"] += 1
    n, t = s["n"], s["step"]
    if s["bits"] == 8 or s["kind"] == "bf16":
        d_m, d_v, d_p = draws(n, s["seed"], t)
    g = s["grad"] * s["grad_scale"]
    m = s["m"] if s["bits"] == 32 else unpack8(s["m"], s["m_exp"], 3)
    v = s["v"] if s["bits"] == 32 else unpack8(s["v"], s["v_exp"], 4).square()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    w = s["param"].float() if s["master"] is None else s["master"]
    w = w * (1 - LR * DECAY) - (LR / (1 - BETA1 ** t)) * m / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        out = {"m": s["m"], "v": s["v"]}
    else:
        s["m"], s["m_exp"] = pack8(m, d_m, 3)
        s["v"], s["v_exp"] = pack8(v.sqrt(), d_v, 4)
        out = {"m": unpack8(s["m"], s["m_exp"], 3).to(BF16), "v": unpack8(s["v"], s["v_exp"], 4).to(BF16)}
    if s["kind"] == "bf16":
        # a bf16 parameter with no master copy is rounded by a draw as well
        s["param"].copy_(((w.view(torch.int32) + d_p) & -65536).view(F32))
    else:
        s["param"].copy_(w)
    if s["master"] is not None:
        out["master"] = s["master"].copy_(w)
    return dict(out, param=s["param"])


# ---------------------------------------------------------------------------
# the framework's calls; what a program keeps between them is made at the first
# ---------------------------------------------------------------------------
def layer(occ, T, d, E, k, n_vdev, dtype):
    ds = occ.occult_desc_t()
    ds.T, ds.d, ds.n_experts, ds.top_k, ds.n_vdev, ds.inter = T, d, E, k, n_vdev, 64
    ds.dtype = occ.OCCULT_BF16 if dtype == "bf16" else occ.OCCULT_F32
    return ds


def norm_handle(s):
    import combine_top_route_gb300 as occ
    desc = layer(occ, s["T"], s["d"], 8, 2, 4, s["dtype"])
    kind = {"none": occ.GATE_NONE, "channel": occ.GATE_CHANNEL, "token": occ.GATE_TOKEN}[s["gate"]]
    opt = occ.occult_norm_t(s["eps"], s["res_scale"], kind,
                            occ.OCCULT_BF16 if s["res"] == "bf16" else occ.OCCULT_F32)
    need = occ.workspace_size(desc, occ.WS_BLOCK_NORM_BWD)
    ws = torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
    s["handle"] = occ, desc, opt, ws
    return s["handle"]


def own_norm(s):
    occ, desc, opt, _ = s.get("handle") or norm_handle(s)
    occ.occult_block_norm(desc, opt, s["r"], y=s["y"], w_post=s["w_post"], gate=s["gate_v"],
                          w_pre=s["w_pre"], r_out=s["r_out"], x=s["x"], rstd_post=s["rstd_post"],
                          rstd_pre=s["rstd_pre"])
    out = {"r_out": s["r_out"]}
    if s["post"]:
        out["rstd_post"] = s["rstd_post"]
    if s["pre"]:
        out.update(rstd_pre=s["rstd_pre"], x=s["x"])
    return out


def own_norm_grad(s):
    occ, desc, opt, ws = s.get("handle") or norm_handle(s)
    occ.occult_block_norm_bwd(desc, opt, s["dr_out"], s["r_out"], s["dr"], ws, dx=s["dx"], y=s["y"],
                              w_post=s["w_post"], gate=s["gate_v"], w_pre=s["w_pre"],
                              rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"], dy=s["dy"],
                              dw_post=s["dw_post"], dgate=s["dgate"], dw_pre=s["dw_pre"])
    out = {"dr": s["dr"], "dy": s["dy"]}
    if s["post"]:
        out["dw_post"] = s["dw_post"]
    if s["pre"]:
        out["dw_pre"] = s["dw_pre"]
    if s["gate"] != "none":
        out["dgate"] = s["dgate"]
    return out


def own_balance(s):
    if "handle" not in s:
        import combine_top_route_gb300 as occ
        desc = layer(occ, s["T"], 64, s["n_experts"], s["top_k"], s["n_vdev"], "bf16")
        opt = occ.occult_balance_t(s["coef"], s["coef_dev"], s["coef_z"], s["group_len"])
        need = occ.balance_workspace_size(desc, opt)
        s["handle"] = occ, desc, opt, torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
    occ, desc, opt, ws = s["handle"]
    occ.occult_balance_loss(desc, opt, s["logits"], s["ids"], s["e2v"], s["counts"], s["grad_w"],
                            s["loss"], ws, mask=s["mask"])
    occ.occult_balance_grad(desc, opt, s["logits"], s["grad_w"], s["dlogits"], mask=s["mask"],
                            dloss=s["dloss"], accumulate=True)
    return {"loss": s["loss"], "counts": s["counts"], "dlogits": s["dlogits"]}


def own_adamw(s):
    if "handle" not in s:
        import combine_top_route_gb300 as occ
        part = lambda t, a, m: None if t is None else t[a:a + m]  # noqa: E731
        blocks = lambda t, a, m: None if t is None else t[a // STATE_BLOCK:(a + m - 1) // STATE_BLOCK + 1]  # noqa: E731
        table = occ.adamw_table([
            dict(param=part(s["param"], a, m), master=part(s["master"], a, m), grad=part(s["grad"], a, m),
                 m=part(s["m"], a, m), v=part(s["v"], a, m), m_exp=blocks(s["m_exp"], a, m),
                 v_exp=blocks(s["v_exp"], a, m), first=a)
            for a, m in zip(s["starts"], s["sizes"])])
        opt = occ.occult_adamw_t(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY,
                                 state_bits=s["bits"], seed=s["seed"],
                                 grad_scale=s["grad_scale"].data_ptr())
        s["handle"] = occ, table, opt
    occ, table, opt = s["handle"]
    s["step"] += 1
    opt.step = s["step"]
    occ.occult_adamw(opt, table)
    out = {"m": s["m"], "v": s["v"]}
    if s["bits"] == 8:
        out = {"m": s["m_val"], "v": s["v_val"]}
        occ.occult_adamw_read(s["m"], s["m_exp"], occ.STATE_M, s["m_val"])
        occ.occult_adamw_read(s["v"], s["v_exp"], occ.STATE_V, s["v_val"])
    if s["master"] is not None:
        out["master"] = s["master"]
    return dict(out, param=s["param"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] in ("norm", "norm_grad"):
        T, d, post, pre = case["T"], case["d"], case["post"], case["pre"]
        lb, rb = (2 if case[k] == "bf16" else 4 for k in ("dtype", "res"))
        gate = {"none": 0, "channel": d, "token": T}[case["gate"]]
        if case["op"] == "norm":
            per = rb + 4 + rb + (lb if pre else 0)
            small = (post + pre) * (d * lb + 4 * T) + 4 * gate
            return {"bytes": T * d * per + small, "flops": T * d * (3 + 4 * post + 4 * pre)}
        per = rb + (4 + rb if pre else 0) + (4 if post or gate else 0) + rb + lb
        small = (post + pre) * (d * lb + 4 * d + 4 * T) + 8 * gate
        return {"bytes": T * d * per + small, "flops": T * d * (3 + 9 * post + 9 * pre + 2 * (gate > 0))}
    if case["op"] == "balance":
        T, E, k = case["T"], case["n_experts"], case["top_k"]
        G = -(-T // (case["group_len"] or T))
        return {"bytes": 12 * T * E + 4 * T * k + T * case["masked"] + 4 * G * E + 4 * E + 16,
                "flops": 14 * T * E + T * k}
    n = sum(sizes_of(case))
    param = {"f32": 8, "bf16_master": 10, "bf16": 4}[case["kind"]]
    # the gradient, the parameter (and its master), and both states in and out; 8-bit
    # states are read out as bf16 values besides
    state = 16 if case["bits"] == 32 else 4 + 4 + 4 / STATE_BLOCK
    return {"bytes": n * (4 + param + state), "flops": n * 15}


# ---------------------------------------------------------------------------
# the same outputs in 64 bits, from the operators' definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": exact_norm, "norm_grad": exact_norm_grad, "balance": exact_balance,
            "adamw": exact_adamw}[case["op"]](s)


def f64(v):
    return None if v is None else v.double()


def exact_norm(s):
    """Rows in slabs: r' = a r + gate * w y / rms(y), x = w r' / rms(r')."""
    T, out = s["T"], {"r_out": []}
    w_post, w_pre, gate = f64(s["w_post"]), f64(s["w_pre"]), f64(s["gate_v"])
    for a in range(0, T, 8192):
        rows = slice(a, min(T, a + 8192))
        b = s["y"][rows].double()
        if s["post"]:
            inv = 1 / torch.sqrt(b.pow(2).sum(1) / s["d"] + s["eps"])
            out.setdefault("rstd_post", []).append(inv)
            b = torch.einsum("td,t,d->td", b, inv, w_post)
        if s["gate"] == "channel":
            b = torch.einsum("td,d->td", b, gate)
        elif s["gate"] == "token":
            b = torch.einsum("td,t->td", b, gate[rows])
        r = s["r"][rows].double() * s["res_scale"] + b
        out["r_out"].append(r)
        if s["pre"]:
            inv = 1 / torch.sqrt(r.pow(2).sum(1) / s["d"] + s["eps"])
            out.setdefault("rstd_pre", []).append(inv)
            out.setdefault("x", []).append(torch.einsum("td,t,d->td", r, inv, w_pre))
    return {k: torch.cat(v) for k, v in out.items()}


def exact_norm_grad(s):
    """The derivative by the chain rule on slabs of rows: with n = v c and
    c = (mean v^2 + eps)^(-1/2) given, dv = c dn - v c^3 <v, dn> / d."""
    T, d = s["T"], s["d"]
    w_post, w_pre, gate = f64(s["w_post"]), f64(s["w_pre"]), f64(s["gate_v"])
    out = {"dr": [], "dy": []}
    sums = {}

    def back(v, c, dn):
        return c * dn - v * c ** 3 * ((v * dn).sum(1, keepdim=True) / d)

    for a in range(0, T, 8192):
        rows = slice(a, min(T, a + 8192))
        D = s["dr_out"][rows].double()
        if s["pre"]:
            v, c, up = s["r_out"][rows].double(), s["rstd_pre"][rows].double()[:, None], s["dx"][rows].double()
            D = D + back(v, c, up * w_pre)
            sums["dw_pre"] = sums.get("dw_pre", 0) + torch.einsum("td,td,tx->d", up, v, c)
        out["dr"].append(D * s["res_scale"])
        y = s["y"][rows].double()
        c = s["rstd_post"][rows].double()[:, None] if s["post"] else 1.0
        n = y * c
        b = n * w_post if s["post"] else n
        G = D
        if s["gate"] == "channel":
            sums["dgate"] = sums.get("dgate", 0) + (D * b).sum(0)
            G = D * gate
        elif s["gate"] == "token":
            out.setdefault("dgate", []).append((D * b).sum(1))
            G = D * gate[rows][:, None]
        if s["post"]:
            sums["dw_post"] = sums.get("dw_post", 0) + (G * n).sum(0)
            G = back(y, c, G * w_post)
        out["dy"].append(G)
    return dict({k: torch.cat(v) for k, v in out.items()}, **sums)


def exact_balance(s):
    T, E, k, G, L = s["T"], s["n_experts"], s["top_k"], s["G"], s["L"]
    mask = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"].bool()
    e2v, dlogits = s["e2v"].long(), s["dlogits"].double()
    on_dev = torch.nn.functional.one_hot(e2v, s["n_vdev"]).double()
    kept = [mask[a * L:(a + 1) * L].nonzero()[:, 0] + a * L for a in range(G)]
    live = max(1, sum(len(t) > 0 for t in kept))
    tokens = max(1, sum(len(t) for t in kept))
    counts = torch.zeros(G, E, dtype=torch.int32, device=DEV)
    bal = dev = sq = 0.0
    for a, t in enumerate(kept):
        if not len(t):
            continue
        z = s["logits"][t].double()
        lse = torch.logsumexp(z, 1)
        p = (z - lse[:, None]).exp()
        c = torch.bincount(s["ids"][t].long().view(-1), minlength=E)
        counts[a] = c
        f, share = c.double() * E / (k * len(t)), p.mean(0)
        f_dev = on_dev.T @ f / on_dev.sum(0)
        bal = bal + f @ share / live
        dev = dev + f_dev @ (on_dev.T @ share) / live
        sq = sq + lse.pow(2).sum() / tokens
        # loss = sum_t h . p_t with constant h: the softmax's Jacobian gives p (h - h . p)
        h = (s["coef"] * f + s["coef_dev"] * f_dev[e2v]) / (live * len(t))
        dz = p * h - p * (p @ h)[:, None] + 2 * s["coef_z"] / tokens * lse[:, None] * p
        dlogits[t] += s["dloss"].double() * dz
    loss = s["coef"] * bal + s["coef_dev"] * dev + s["coef_z"] * sq
    return {"loss": torch.stack([torch.as_tensor(x, dtype=torch.float64, device=DEV) for x in (loss, bal, dev, sq)]),
            "counts": counts, "dlogits": dlogits}


def hash32(x):
    """Multiply, fold the high 17 bits in, multiply, fold the high half in: all mod 2^32."""
    a = x % (1 << 32) * MUL1 % (1 << 32)
    b = (a ^ (a // (1 << 15))) * MUL2 % (1 << 32)
    return b ^ (b // (1 << 16))


def exact_adamw(s):
    """On slabs of whole blocks.  A code stands for c * 2^(E - 15 - mantissa bits) with
    E the block's exponent; the rounding is floor(x / unit + draw / 2^16)."""
    n, t = s["n"], s["step"] + 1
    key = hash32(s["seed"] + hash32(t))
    scale = s["grad_scale"].double()
    out = {"m": [], "v": [], "param": []}

    def value(code, exp, mant):
        e = exp.double().repeat_interleave(STATE_BLOCK) - 15 - 127
        mag = (code.int() % (16 << mant)).double()
        oct_, frac = torch.floor(mag / (1 << mant)), mag % (1 << mant)
        x = torch.where(mag > 0, (1 + frac / (1 << mant)) * torch.exp2(oct_ + e), 0.0)
        return torch.where(code >= 128, -x, x) if mant == 3 else x

    def rounded(x, u, mant):
        mag = x.abs()
        top = mag.view(-1, STATE_BLOCK).amax(1)
        fr, ex = torch.frexp(top)  # top = fr 2^ex, fr in [1/2, 1): the binade above if rounding up reaches it
        emax = torch.where(fr * (2 << mant) > (2 << mant) - 1, ex + 1, ex) - 1
        emax = emax.clamp(min=16 - 127).repeat_interleave(STATE_BLOCK)
        unit = torch.exp2((torch.frexp(mag)[1] - 1 - mant).double())
        q = torch.floor(mag / unit + u) * unit
        low = torch.exp2((emax - 15).double())  # codes run from just above this
        if mant == 3:
            q = torch.where(q > low, q, 0.0)
        else:
            q = torch.where((q > low) | (mag == 0), q, low * (1 + 1 / 16))
        return torch.where(mag > 0, torch.sign(x) * q, 0.0)

    for a in range(0, n, 1 << 26):
        i = slice(a, min(n, a + (1 << 26)))
        blocks = slice(a // STATE_BLOCK, -(-i.stop // STATE_BLOCK))
        g = s["grad"][i].double() * scale
        small = s["bits"] == 8
        m = value(s["m"][i], s["m_exp"][blocks], 3) if small else s["m"][i].double()
        v = value(s["v"][i], s["v_exp"][blocks], 4) ** 2 if small else s["v"][i].double()
        m, v = m + (1 - BETA1) * (g - m), v + (1 - BETA2) * (g ** 2 - v)
        w = (s["param"] if s["master"] is None else s["master"])[i].double()
        mean, second = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
        w = w - LR * DECAY * w - LR * mean / (second.sqrt() + EPS)
        r = hash32(torch.arange(i.start, i.stop, device=DEV) + key)
        if small:
            out["m"].append(rounded(m, (r % 65536) / 65536, 3).float())
            out["v"].append(rounded(v.sqrt(), torch.div(r, 65536, rounding_mode="floor") / 65536, 4).float())
        else:
            out["m"].append(m)
            out["v"].append(v)
        if s["master"] is not None:
            out.setdefault("master", []).append(w)
        if s["kind"] == "bf16":
            unit = torch.exp2((torch.frexp(w)[1] - 8).double())
            u = torch.div((r * MUL1) & M32, 65536, rounding_mode="floor") / 65536
            w = torch.sign(w) * torch.floor(w.abs() / unit + u) * unit
            w = torch.where(torch.isfinite(w), w, 0.0)
        out["param"].append(w)
    return {k: torch.cat([x.double() for x in v]) for k, v in out.items()}
