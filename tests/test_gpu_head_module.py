"""OccultHead in the forms that a model uses it in, and the chain under a softmax router.

Gradients against fp64 autograd of the same formulas.  bf16: the tolerance of the chain's other
tests (2-norm of the difference over that of the gradient, some twenty roundings to bf16 of
2^-9 / sqrt(3) each, amplified by the norms: 1.5 %).  fp32: products of up to 300 terms, each
within 2^-24, twice over, and the norm's: 1e-4 of the 2-norm; bf16 residual streams round
dr once, 2^-8.
"""
import os
import sys

import numpy as np
import pytest
import torch

import synth

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

REL = 0.015


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


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def rms(v):
    return v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt()


def head_total(o, z, labels, teacher):
    """The head's total in fp64, from the logits."""
    lse = z.logsumexp(1)
    on = torch.zeros_like(lse, dtype=torch.bool)
    total = 0.0
    if labels is not None:
        on = labels >= 0
        total = total + o.coef * (lse - z.gather(1, labels.clamp(min=0).long()[:, None])[:, 0])[on].mean()
    if teacher is not None:
        ids, tl = teacher
        q, logp = (tl.double() / o.temperature).softmax(1), (z / o.temperature).log_softmax(1).gather(1, ids.long())
        total = total + o.coef_kd * o.temperature ** 2 * (q * (q.log() - logp)).sum(1).mean()
        on = torch.ones_like(on)
    return total + o.coef_z * lse[on].square().mean()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("biased", [True, False])
def test_gradients_of_the_chain_under_a_softmax_router(occ, renorm, biased):
    from train_model import Model, batch
    cfg = synth.CONFIGS["olmoe_train"].with_(name="model", T=384, d=128, inter=64, n_experts=8, top_k=2, n_vdev=4,
                                             renorm=renorm)
    model = Model(cfg, 500, coef=0.8, coef_z=1e-2)
    block, head, moe = model.block, model.head, model.block.moe
    moe.score.score, moe.score.scale = occ.SCORE_SOFTMAX, 2.0
    for name in ("w1", "w2"):
        moe.w[name].mul_(4)      # activations of order one in a layer this narrow
    g = torch.Generator(device="cuda").manual_seed(5)
    moe.bias = 0.05 * torch.randn(8, generator=g, device="cuda") if biased else None
    pairs, labels, _ = batch(cfg, 500, 1, 0)
    labels[::5] = -100
    losses = model.gradients(pairs, labels)
    p = {n: t.detach().double().requires_grad_() for n, t, _ in model.parameters()}
    r = model.stream(pairs).double().requires_grad_()
    x = rms(r) * p["w_pre"]
    logits = x @ p["w_router"].T
    ids = moe.ids.long()
    gates = logits.softmax(1).gather(1, ids)
    gates = 2.0 * (gates / gates.sum(1, keepdim=True) if renorm else gates)
    y = torch.zeros_like(x)
    for e in range(8):
        rows, slot = (ids == e).nonzero(as_tuple=True)
        w1, w2 = p["w1"].view(8, 128, 128)[e], p["w2"].view(8, 128, 64)[e]
        h = torch.nn.functional.silu(x[rows] @ w1[:64].T) * (x[rows] @ w1[64:].T)
        y = y.index_add(0, rows, gates[rows, slot][:, None] * (h @ w2.T))
    out = r + p["gate"] * (rms(y) * p["w_post"])
    total = head_total(head.opt, (rms(out) * p["w_norm"]) @ p["w_head"].T, labels, None)
    (total + block.bal_opt.coef_z * logits.logsumexp(1).square().mean()).backward()
    torch.cuda.synchronize()
    assert abs(float(losses[0]) / float(total.detach()) - 1) < REL
    assert rel(block.dr, r.grad) < REL
    for name, _, grad in model.parameters():
        assert rel(grad.view_as(p[name].grad), p[name].grad) < REL, name


def fp32_head(occ, T=200, d=64, V=300, res=torch.float32, **kw):
    desc = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=T, d=d, dtype="f32"))
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(V, d, generator=g, device="cuda") / 8
    head = occ.OccultHead(desc, w, res_dtype=res, **kw)
    head.w_norm.copy_(1 + 0.2 * torch.randn(d, generator=g, device="cuda"))
    r = torch.randn(T, d, generator=g, device="cuda").to(res)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    labels[::6] = -1
    ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:4] for _ in range(T)]).int()
    return head, r, labels, (ids, torch.randn(T, 4, generator=g, device="cuda"))


@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("taught", [False, True])
def test_head_of_an_fp32_layer(occ, res, taught):
    kw = dict(coef=0.6, coef_z=1e-2)
    if taught:
        kw.update(topk=4, coef_kd=0.5, temperature=2.0)
    head, r, labels, teacher = fp32_head(occ, res=res, **kw)
    teacher = teacher if taught else None
    up = torch.full((1,), 0.25, device="cuda")
    losses, dr = head.step(r, labels, teacher, dloss=up)
    p = {n: t.detach().double().requires_grad_() for n, t, _ in head.parameters()}
    x = r.double().requires_grad_()
    total = head_total(head.opt, (rms(x) * p["w_norm"]) @ p["w_head"].T, labels, teacher)
    (0.25 * total).backward()
    torch.cuda.synchronize()
    assert abs(float(losses[0]) / float(total.detach()) - 1) < 1e-5
    assert rel(dr, x.grad) < (1e-4 if res == torch.float32 else 2.0 ** -8)
    for name, _, grad in head.parameters():
        assert rel(grad, p[name].grad) < 1e-4, name
    again = head.loss(r, labels, teacher)
    assert abs(float(again[0]) / float(total.detach()) - 1) < 1e-5


def test_token_losses_are_of_the_last_call(occ):
    """A call without labels leaves no other call's token losses behind."""
    head, r, labels, teacher = fp32_head(occ, topk=4, coef=0.5, coef_kd=0.5)
    for call in (head.step, head.loss):
        head.loss(r, labels, teacher)
        assert (head.token_loss[labels >= 0] > 0).all()
        call(r, None, teacher)
        assert (head.token_loss == 0).all()
        assert (head.lse != 0).all()


def test_bias_step_before_any_forward(occ):
    """No loads yet: the bias stays."""
    cfg = synth.CONFIGS["olmoe_train"].with_(T=64, d=128, inter=64, n_experts=8, top_k=2, n_vdev=4)
    held = [torch.full((n,), 7 * i, dtype=torch.int32, device="cuda") for i in range(1, 400) for n in (8, 128)]
    for t in held:
        t[0] = 1000
    torch.cuda.synchronize()
    del t, held          # what freshly allocated memory then holds
    block = occ.OccultBlock(occ.desc_for(cfg), synth.expert_weights(cfg, device="cuda"),
                            torch.arange(8, dtype=torch.int32).view(4, 2), torch.zeros(8, 128),
                            score=occ.occult_score_t(bias_rate=0.5), bias=torch.zeros(8))
    block.bias_step()
    assert (block.moe.bias == 0).all() and (block.counts == 0).all()


def test_a_head_that_only_scores(occ):
    """train=False: no gradients and no kept logits; the same losses; a step is refused."""
    desc = occ.desc_for(synth.CONFIGS["olmoe_fwd"].with_(T=300, d=128))
    g = torch.Generator(device="cuda").manual_seed(2)
    w = (torch.randn(4000, 128, generator=g, device="cuda") / 8).bfloat16()
    r = torch.randn(300, 128, generator=g, device="cuda").bfloat16()
    labels = torch.randint(0, 4000, (300,), generator=g, device="cuda").int()
    full, lean = occ.OccultHead(desc, w), occ.OccultHead(desc, w, train=False)
    a, b = full.loss(r, labels).clone(), lean.loss(r, labels)
    assert torch.equal(a, b) and torch.equal(full.token_loss, lean.token_loss)
    assert lean.dw is None and lean.dx is None
    assert lean.ws.numel() == occ.head_workspace_size(desc, lean.opt, step=False) < full.ws.numel()
    with pytest.raises(RuntimeError, match="train=True"):
        lean.step(r, labels)
    with pytest.raises(RuntimeError, match="train=True"):
        lean.parameters()
