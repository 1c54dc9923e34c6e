"""Workloads of a model's two choices next to the MoE layer: experts and next tokens.

Three operators and their cases: the scored router (softmax or sigmoid scores, a
bias that evens out the loads, groups of experts, with its gradient), the loss of
the output head (softmax cross entropy over a large vocabulary, with its
gradients) and distillation from a teacher's top logits through the same head.
``run`` makes one pass of an operator: in its plain form (elementary torch
operations in fp32, the router's scores in fp64) or, with ``own`` set, through
``combine_top_route_gb300``.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
OFF = torch.finfo(F32).min   # a logit as low as this switches its expert off


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token choosing 8 of 64 experts; latency is all that counts
        route("route_one_token", 1, 64, 8, 8, "sigmoid", 1, 1, 1, "blocks", True, True, False),
        # 512 concurrent decode tokens, 4 of 8 groups, some experts switched off
        route("route_decode_512", 512, 256, 8, 8, "sigmoid", 8, 4, 2, "blocks", True, True, False,
              off=0.05),
        # a training step's 32768 tokens over 256 experts in 8 groups, and the gradient
        route("route_train", 32768, 256, 8, 8, "sigmoid", 8, 4, 2, "blocks", True, True, True),
        # prefill-shaped softmax routing limited to 2 of 4 devices, an odd number of tokens
        route("route_devices_odd", 16383, 60, 4, 4, "softmax", 4, 2, 1, "vdev", False, False, True),
        # one token scored in decoding: its log-probability under the whole vocabulary
        head("loss_one_token", False, 1, 2048, 50304, "bf16", coef=1.0),
        # an evaluation batch: the loss alone
        head("loss_eval", False, 4096, 2048, 50304, "bf16", coef=1.0),
        # the small fp32 layer's head with an odd vocabulary
        head("loss_train_f32_small", True, 257, 64, 1009, "f32", coef=1.0, coef_z=1e-4, ignored=0.1),
        # a training step's head: loss, z term and both gradients
        head("loss_train", True, 8192, 2048, 50304, "bf16", coef=1.0, coef_z=1e-4),
        # fine-tuning on answers alone: 3 of 5 tokens ignored, odd sizes
        head("loss_finetune_ragged", True, 4095, 2048, 102401, "bf16", coef=1.0, ignored=0.6),
        # scoring a student against a teacher's top 32 logits, no labels
        head("distill_eval", False, 2048, 2048, 151936, "bf16", topk=32, coef_kd=1.0, temperature=1.0),
        # a small batch of a fine-tuning after pruning, the unpruned model as the teacher
        head("distill_small", True, 129, 512, 32000, "bf16", topk=8, coef_kd=1.0, temperature=2.0),
        # a training step on labels and a teacher's top 64 logits
        head("distill_train", True, 4096, 2048, 50304, "bf16", topk=64, coef=0.5, coef_kd=0.5,
             temperature=2.0, ignored=0.1),
    ]


def route(name, T, n_experts, top_k, n_vdev, score, groups, keep, best, kind, bias, renorm, grad,
          off=0.0):
    return {"name": name, "op": "route", "T": T, "n_experts": n_experts, "top_k": top_k,
            "n_vdev": n_vdev, "score": score, "groups": groups, "keep": keep, "best": best,
            "kind": kind, "bias": bias, "renorm": renorm, "grad": grad, "off": off}


def head(name, grad, T, d, vocab, dtype, topk=0, coef=0.0, coef_kd=0.0, coef_z=0.0, temperature=1.0,
         ignored=0.0):
    return {"name": name, "op": "head", "grad": grad, "T": T, "d": d, "vocab": vocab, "dtype": dtype,
            "topk": topk, "coef": coef, "coef_kd": coef_kd, "coef_z": coef_z,
            "temperature": temperature, "ignored": ignored}


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.4:
        n_vdev = rng.choice([1, 2, 4, 8, 16])
        per = rng.randint(max(1, 8 // n_vdev), 256 // n_vdev)
        E = n_vdev * per
        kind = rng.choice(["blocks", "blocks", "vdev"])
        groups = n_vdev if kind == "vdev" else rng.choice([g for g in (1, 1, 2, 3, 4, 8) if E % g == 0])
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * (E // groups)))
        c = route("", log_int(rng, 1, 32768), E, k, n_vdev, rng.choice(["sigmoid", "sigmoid", "softmax"]),
                  groups, keep, rng.choice([1, 2]), kind, rng.random() < 0.7, rng.random() < 0.7,
                  rng.random() < 0.5, off=rng.choice([0.0, 0.0, 0.1]))
    elif rng.random() < 0.15:
        T, d = log_int(rng, 1, 700), 64 * rng.randint(1, 4)
        c = head("", rng.random() < 0.7, T, d, log_int(rng, 16, 4001), "f32", topk=rng.choice([0, 5]),
                 coef=1.0, coef_kd=0.5, coef_z=rng.choice([0.0, 1e-4]), temperature=1.5,
                 ignored=rng.choice([0.0, 0.3]))
    else:
        d = 64 * log_int(rng, 1, 64)
        vocab = log_int(rng, 500, 152000)
        T = log_int(rng, 1, min(16384, 8192 * 2048 * 50304 // (2 * d * vocab)))
        topk = rng.choice([0, 0, 1, 16, 64, 100])
        coef = rng.choice([0.0, 1.0, 0.3]) if topk else 1.0
        c = head("", rng.random() < 0.6, T, d, vocab, "bf16", topk=topk, coef=coef,
                 coef_kd=1.0 - coef if coef < 1 else 0.5 * bool(topk), coef_z=rng.choice([0.0, 1e-4]),
                 temperature=rng.choice([1.0, 2.0, 0.7, 4.0]) if topk else 1.0,
                 ignored=rng.choice([0.0, 0.0, 0.2, 0.8]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return prepare_route(case, g) if case["op"] == "route" else prepare_head(case, g)


def prepare_route(case, g):
    T, E, k, n_vdev = case["T"], case["n_experts"], case["top_k"], case["n_vdev"]
    randn = lambda *n: torch.randn(*n, generator=g, device=DEV)  # noqa: E731
    s = dict(case, scale=2.5 if case["renorm"] else 1.0)
    # tokens of 16 latent clusters, each drawn to a sixth of the experts
    likes = (torch.rand(16, E, generator=g, device=DEV) < 1 / 6).float()
    cluster = torch.randint(0, 16, (T,), generator=g, device=DEV)
    s["logits"] = randn(T, E) + 3 * likes[cluster] - 1.5
    if case["off"]:
        gone = torch.rand(T, E, generator=g, device=DEV) < case["off"]
        s["logits"] = s["logits"].masked_fill(gone, -math.inf)
    # a bias moved in steps of a thousandth
    s["bias"] = 1e-3 * torch.randint(-60, 61, (E,), generator=g, device=DEV).float() if case["bias"] else None
    # a placement that deals the experts out at random
    s["e2v"] = (torch.randperm(E, generator=g, device=DEV) % n_vdev).to(I32)
    s["dgates"] = randn(T, k)
    s["ids"], s["vmask"] = (torch.empty(*n, dtype=I32, device=DEV) for n in ((T, k), (T,)))
    s["gates"], s["dlogits"] = (torch.empty(*n, device=DEV) for n in ((T, k), (T, E)))
    return s


def prepare_head(case, g):
    T, d, V, K = case["T"], case["d"], case["vocab"], case["topk"]
    dt = BF16 if case["dtype"] == "bf16" else F32
    randn = lambda *n: torch.randn(*n, generator=g, device=DEV)  # noqa: E731
    randint = lambda lo, hi, *n: torch.randint(lo, hi, n, generator=g, device=DEV)  # noqa: E731
    s = dict(case)
    s["w"] = (1.8 / d ** 0.5 * randn(V, d)).to(dt)
    right = randint(0, V, T)
    # normed rows that lean towards the right token's row, as a trained model's do
    lean = s["w"][right].float()
    s["x"] = (randn(T, d) + 5.0 * lean / lean.norm(dim=1, keepdim=True)).to(dt)
    out = torch.rand(T, generator=g, device=DEV) < case["ignored"]
    s["labels"] = torch.where(out, -100, right).to(I32) if case["coef"] else None
    s["t_ids"] = s["t_logits"] = None
    if K:
        # distinct tokens, the right one first; a few rows with fewer than K
        step = 1 + torch.rand(T, 1, generator=g, device=DEV) * max(0, (V - 1) // K - 1)
        j = torch.arange(K, device=DEV)
        ids = (right[:, None] + j * step.long()) % V
        logits = randn(T, K).sort(dim=1, descending=True).values * 1.5 + 14
        logits[:, 0] += 2.0
        short = torch.rand(T, 1, generator=g, device=DEV) < 0.1
        ids = torch.where(short & (j > K // 2) | out[:, None], -1, ids)
        s["t_ids"], s["t_logits"] = ids.to(I32).contiguous(), logits.contiguous()
    s["dloss"] = torch.ones(1, device=DEV)
    s["loss"], s["lse"], s["token_loss"] = (torch.empty(n, device=DEV) for n in (4, T, T))
    if case["grad"]:
        s["dx"], s["dw"] = torch.empty(T, d, dtype=dt, device=DEV), torch.empty(V, d, dtype=dt, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if s["op"] == "route":
        return own_route(s) if own else plain_route(s)
    return own_head(s) if own else plain_head(s)


def plain_route(s):
    """The scored router; its ranks in fp64, so that near ties fall as the formula says."""
    T, E, k, G = s["T"], s["n_experts"], s["top_k"], s["groups"]
    z = s["logits"]
    off = z <= OFF
    z64 = z.double()
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-z64))
    else:
        top = z64.masked_fill(off, -math.inf).amax(dim=1, keepdim=True)
        score = torch.exp(z64 - torch.where(top.isinf(), 0.0, top)).masked_fill(off, 0.0)
        total = score.sum(dim=1, keepdim=True)
        score = score / torch.where(total == 0, 1.0, total)
    score = score.masked_fill(off, 0.0)
    biased = score if s["bias"] is None else score + s["bias"].double()
    rank = z64 if s["bias"] is None else biased
    rank = rank.masked_fill(off, -1e300)
    if G > 1:
        group = s["e2v"].long() if s["kind"] == "vdev" else torch.arange(E, device=DEV) // (E // G)
        members = torch.sort(group, stable=True).indices.view(G, E // G)
        inside = biased.masked_fill(off, -math.inf)[:, members]
        best = torch.sort(inside, dim=2, descending=True).values[:, :, :s["best"]]
        worth = torch.where(best.isinf(), 0.0, best).sum(dim=2)
        worth = torch.where(best[:, :, 0].isinf(), -math.inf, worth)
        kept = torch.sort(worth, dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        use = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        rank = rank.masked_fill(~use[:, group], -math.inf)
    ids = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = score.gather(1, ids)
    total = chosen.sum(dim=1, keepdim=True)
    total = torch.where(total == 0, 1.0, total)
    share = chosen / total
    gates = s["scale"] * (share if s["renorm"] else chosen)
    bits = torch.zeros(T, s["n_vdev"], dtype=torch.int64, device=DEV)
    bits.scatter_(1, s["e2v"].long()[ids], 1)
    vmask = (bits << torch.arange(s["n_vdev"], device=DEV)).sum(dim=1)
    out = {"ids": s["ids"].copy_(ids), "gates": s["gates"].copy_(gates), "vmask": s["vmask"].copy_(vmask)}
    if not s["grad"]:
        return out
    up = s["scale"] * s["dgates"].double()
    dscore = (up - (up * share).sum(dim=1, keepdim=True)) / total if s["renorm"] else up
    if s["score"] == "sigmoid":
        dz = torch.zeros_like(z64).scatter_(1, ids, dscore * chosen * (1 - chosen))
    else:
        dz = torch.zeros_like(z64).scatter_(1, ids, dscore * chosen)
        dz -= score * (dscore * chosen).sum(dim=1, keepdim=True)
    return dict(out, dlogits=s["dlogits"].copy_(dz))


def teacher(s, V):
    """The teacher's probabilities over its top entries, zero where there is none."""
    valid = (s["t_ids"] >= 0) & (s["t_ids"] < V)
    t = (s["t_logits"] / s["temperature"]).masked_fill(~valid, -math.inf)
    top = t.amax(dim=1, keepdim=True)
    q = torch.exp(t - torch.where(top.isinf(), 0.0, top))
    total = q.sum(dim=1, keepdim=True)
    q = q / torch.where(total == 0, 1.0, total)
    return valid[:, 0], torch.where(valid, s["t_ids"], 0).long(), q


def plain_head(s):
    """Cross entropy, distillation and z term of the head, and the gradients of x and w."""
    V, tau, dt = s["vocab"], s["temperature"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    no = torch.zeros(s["T"], dtype=torch.bool, device=DEV)
    ce_on = no if s["labels"] is None else (s["labels"] >= 0) & (s["labels"] < V)
    kd_on, t_ids, q = (no, None, None) if s["t_ids"] is None else teacher(s, V)
    on = ce_on | kd_on
    n_ce, n_kd, n = (m.sum().clamp(min=1).float() for m in (ce_on, kd_on, on))
    top = z.amax(dim=1, keepdim=True)
    lse = (top + torch.log(torch.exp(z - top).sum(dim=1, keepdim=True))).squeeze(1)
    lse = torch.where(on, lse, 0.0)
    zero = torch.zeros((), device=DEV)
    label = None if s["labels"] is None else torch.where(ce_on, s["labels"], 0).long()
    token = None if label is None else torch.where(ce_on, lse - z.gather(1, label[:, None])[:, 0], 0.0)
    ce = zero if token is None else token.sum() / n_ce
    kd = zero
    if q is not None:
        lse_t = (top / tau + torch.log(torch.exp((z - top) / tau).sum(dim=1, keepdim=True)))
        gap = torch.log(torch.where(q > 0, q, 1.0)) - (z.gather(1, t_ids) / tau - lse_t)
        kd = tau * tau * torch.where(kd_on[:, None] & (q > 0), q * gap, 0.0).sum() / n_kd
    z_term = (lse * lse).sum() / n
    total = s["coef"] * ce + s["coef_kd"] * kd + s["coef_z"] * z_term
    out = {"loss": s["loss"].copy_(torch.stack([total, ce, kd, z_term])), "lse": s["lse"].copy_(lse)}
    if token is not None:
        out["token_loss"] = s["token_loss"].copy_(token)
    if not s["grad"]:
        return out
    a = torch.where(ce_on, s["coef"] / n_ce, zero) + torch.where(on, 2 * s["coef_z"] * lse / n, zero)
    dz = torch.exp(z - torch.where(on, lse, math.inf)[:, None]) * a[:, None]
    if label is not None:
        dz.scatter_add_(1, label[:, None], torch.where(ce_on, -s["coef"] / n_ce, zero)[:, None])
    if q is not None:
        b = torch.where(kd_on, s["coef_kd"] * tau / n_kd, zero)[:, None]
        dz += torch.exp(z / tau - lse_t) * b
        dz.scatter_add_(1, t_ids, -b * q)
    dz *= s["dloss"]
    return dict(out, dx=s["dx"].copy_(dz @ w), dw=s["dw"].copy_(dz.t() @ x))


# ---------------------------------------------------------------------------
# the framework's calls; what a program keeps between them is made at the first
# ---------------------------------------------------------------------------
def layer(occ, T, d, E, k, n_vdev, dtype, renorm=False):
    ds = occ.occult_desc_t()
    ds.T, ds.d, ds.n_experts, ds.top_k, ds.n_vdev, ds.inter = T, d, E, k, n_vdev, 64
    ds.dtype, ds.renorm = (occ.OCCULT_BF16 if dtype == "bf16" else occ.OCCULT_F32), int(renorm)
    return ds


def own_route(s):
    if "handle" not in s:
        import combine_top_route_gb300 as occ
        desc = layer(occ, s["T"], 64, s["n_experts"], s["top_k"], s["n_vdev"], "bf16", s["renorm"])
        opt = occ.occult_score_t(
            score=occ.SCORE_SIGMOID if s["score"] == "sigmoid" else occ.SCORE_SOFTMAX,
            n_groups=s["groups"], keep_groups=s["keep"], group_best=s["best"],
            group_kind=occ.GROUP_VDEV if s["kind"] == "vdev" else occ.GROUP_BLOCKS, scale=s["scale"])
        s["handle"] = occ, desc, opt
    occ, desc, opt = s["handle"]
    occ.occult_route_scored(desc, opt, s["logits"], s["e2v"], s["ids"], s["gates"], s["vmask"],
                            bias=s["bias"])
    out = {"ids": s["ids"], "gates": s["gates"], "vmask": s["vmask"]}
    if s["grad"]:
        occ.occult_route_scored_grad(desc, opt, s["logits"], s["ids"], s["dgates"], s["dlogits"])
        out["dlogits"] = s["dlogits"]
    return out


def own_head(s):
    if "handle" not in s:
        import combine_top_route_gb300 as occ
        desc = layer(occ, s["T"], s["d"], 8, 2, 4, s["dtype"])
        opt = occ.occult_head_t(
            vocab=s["vocab"], topk=s["topk"], coef=s["coef"], coef_kd=s["coef_kd"],
            coef_z=s["coef_z"], temperature=s["temperature"],
            grad_dtype=occ.OCCULT_BF16 if s["dtype"] == "bf16" else occ.OCCULT_F32)
        need = occ.head_workspace_size(desc, opt, step=s["grad"])
        s["handle"] = occ, desc, opt, torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
    occ, desc, opt, ws = s["handle"]
    token = None if s["labels"] is None else s["token_loss"]
    out = {"loss": s["loss"], "lse": s["lse"]}
    if token is not None:
        out["token_loss"] = token
    if not s["grad"]:
        occ.occult_head_loss(desc, opt, s["x"], s["w"], s["loss"], ws, labels=s["labels"],
                             teacher_ids=s["t_ids"], teacher_logits=s["t_logits"], lse=s["lse"],
                             token_loss=token)
        return out
    occ.occult_head_step(desc, opt, s["x"], s["w"], s["loss"], ws, dx=s["dx"], dw=s["dw"],
                         labels=s["labels"], teacher_ids=s["t_ids"], teacher_logits=s["t_logits"],
                         dloss=s["dloss"], lse=s["lse"], token_loss=token)
    return dict(out, dx=s["dx"], dw=s["dw"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k, grad = case["n_experts"], case["top_k"], case["grad"]
        # the choice of k as one comparison for every expert and slot of a tournament
        return {"bytes": 4 * T * E * (1 + grad) + T * k * (8 + 4 * grad) + 4 * T + 8 * E,
                "flops": T * E * (8 + 4 * grad) + T * k * 8}
    d, V, K = case["d"], case["vocab"], case["topk"]
    size = 2 if case["dtype"] == "bf16" else 4
    n = max(1, round(T * (1 - case["ignored"])))   # rows of ignored tokens need no work
    return {"bytes": (n + V) * d * size + case["grad"] * (T + V) * d * size + T * (12 + 8 * K),
            "flops": n * V * (d * 2 * (3 if case["grad"] else 1) + 4)}


# ---------------------------------------------------------------------------
# the same outputs in 64 bits, from the operators' definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return exact_route(s) if case["op"] == "route" else exact_head(s)


def exact_route(s):
    z = s["logits"].double().cpu().numpy()
    T, E = z.shape
    rows, k, G = np.arange(T)[:, None], s["top_k"], s["groups"]
    off = z <= float(OFF)
    with np.errstate(over="ignore", invalid="ignore"):
        if s["score"] == "sigmoid":
            p = np.where(off, 0.0, 1 / (1 + np.exp(-z)))
        else:
            e = np.exp(np.where(off, -np.inf, z - np.max(np.where(off, -1e300, z), axis=1, keepdims=True)))
            p = e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)
    b = 0.0 if s["bias"] is None else s["bias"].double().cpu().numpy()
    key = z if s["bias"] is None else p + b
    level = np.where(off, 1, 0)   # 0: a choice, 1: switched off, 2: in no kept group
    if G > 1:
        group = s["e2v"].cpu().numpy() if s["kind"] == "vdev" else np.arange(E) // (E // G)
        worth = np.empty((T, G))
        for g in range(G):
            mine = np.where(off, -np.inf, p + b)[:, group == g]
            first = -np.sort(-mine, axis=1)[:, :s["best"]]
            worth[:, g] = np.where(first[:, 0] == -np.inf, -np.inf, np.where(first == -np.inf, 0, first).sum(axis=1))
        place = np.argsort(np.argsort(-worth, axis=1, kind="stable"), axis=1, kind="stable")
        level = np.where(place[:, group] < s["keep"], level, 2)
    key = np.where(level > 0, 0.0, key)
    ids = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -key, level), axis=1)[:, :k]
    c = p[rows, ids]
    total = c.sum(axis=1, keepdims=True)
    total = np.where(total == 0, 1.0, total)
    gates = s["scale"] * (c / total if s["renorm"] else c)
    out = {"ids": None, "gates": torch.from_numpy(gates), "vmask": None}
    if s["grad"]:
        dg = s["dgates"].double().cpu().numpy()
        # sum over the gates of dgate times gate's derivative by each chosen score
        ds = s["scale"] * (dg / total - (dg * c).sum(axis=1, keepdims=True) / total ** 2) if s["renorm"] else s["scale"] * dg
        full = np.zeros((T, E))
        full[rows, ids] = ds
        dz = full * p * (1 - p) if s["score"] == "sigmoid" else p * (full - (full * p).sum(axis=1, keepdims=True))
        out["dlogits"] = torch.from_numpy(dz)
    return out


def exact_head(s):
    T, V, K, tau = s["T"], s["vocab"], s["topk"], s["temperature"]
    if T * V * s["d"] * (6 if s["grad"] else 2) > 1.5e13:
        return None
    x, w = s["x"].double(), s["w"].double()
    z = torch.mm(x, w.T)
    rows = torch.arange(T, device=DEV)
    target = torch.zeros(T, V, dtype=F64, device=DEV) if s["grad"] else None
    ce_rows = rows[:0] if s["labels"] is None else rows[(s["labels"] >= 0) & (s["labels"] < V)]
    kd_rows = rows[:0] if s["t_ids"] is None else rows[(s["t_ids"][:, 0] >= 0) & (s["t_ids"][:, 0] < V)]
    on = torch.unique(torch.cat([ce_rows, kd_rows]))
    weight = lambda n: 1.0 / max(1, n)  # noqa: E731
    lse = torch.zeros(T, dtype=F64, device=DEV)
    lse[on] = torch.logsumexp(z[on], dim=1)
    token, ce, kd = None, 0.0, 0.0
    if s["labels"] is not None:
        token = torch.zeros(T, dtype=F64, device=DEV)
        right = s["labels"].long()[ce_rows]
        token[ce_rows] = lse[ce_rows] - z[ce_rows, right]
        ce = float(token.sum()) * weight(len(ce_rows))
        if s["grad"]:
            target[ce_rows, right] += s["coef"] * weight(len(ce_rows))
    if K:
        zk, ids, tl = z[kd_rows] / tau, s["t_ids"].long()[kd_rows], s["t_logits"].double()[kd_rows]
        logp = zk - torch.logsumexp(zk, dim=1, keepdim=True)
        there = (ids >= 0) & (ids < V)
        logq = torch.log_softmax(torch.where(there, tl / tau, -math.inf), dim=1)
        q = logq.exp()
        terms = q * (logq - logp.gather(1, ids.clamp(0, V - 1)))
        kd = tau ** 2 * float(torch.where(there, terms, 0.0).sum()) * weight(len(kd_rows))
        if s["grad"]:
            target.index_put_((kd_rows[:, None].expand_as(ids)[there], ids[there]),
                              s["coef_kd"] * tau * weight(len(kd_rows)) * q[there], accumulate=True)
    zz = float((lse ** 2).sum()) * weight(len(on))
    total = s["coef"] * ce + s["coef_kd"] * kd + s["coef_z"] * zz
    out = {"loss": torch.tensor([total, ce, kd, zz], dtype=F64), "lse": lse}
    if token is not None:
        out["token_loss"] = token
    if not s["grad"]:
        return out
    dz = torch.zeros(T, V, dtype=F64, device=DEV)
    part = 2 * s["coef_z"] * weight(len(on)) * lse[on]
    dz[on] += part[:, None] * torch.softmax(z[on], dim=1)
    dz[ce_rows] += s["coef"] * weight(len(ce_rows)) * torch.softmax(z[ce_rows], dim=1)
    if K:
        dz[kd_rows] += s["coef_kd"] * tau * weight(len(kd_rows)) * logp.exp()
    dz = (dz - target) * float(s["dloss"])
    return dict(out, dx=torch.mm(dz, w), dw=torch.mm(dz.T, x))
