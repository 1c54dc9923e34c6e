"""The layer with the scored router, and the router, block, head and update in a row.

Gradients against fp64 autograd of the same formulas with the routing as the block chose
it.  Tolerance (2-norm of the difference over that of the gradient): as the block's own,
some twenty roundings to bf16 of 2^-9 / sqrt(3) each in the 2-norm, two more for the
gradient of the logits and the last norm's output: < 0.7 %; 1.5 % leaves room for the
amplification by the norms.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import synth
from oracle import expert as oexpert
from oracle import scored

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

REL = 0.015
VOCAB = 500


@pytest.fixture(scope="module")
def occ():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_top_route_gb300 import build
    build.build()
    import combine_top_route_gb300 as occ
    occ.lib()
    return occ


def config(**kw):
    return synth.CONFIGS["olmoe_train"].with_(**{**dict(name="model", T=384, d=128, inter=64, n_experts=8,
                                                        top_k=2, n_vdev=4, renorm=True), **kw})


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("merge", ["atomic", "ordered"])
def test_layer_output_by_scores(occ, sigmoid, merge):
    from layer_cases import assert_close_layer, make_case
    cfg = synth.CONFIGS["olmoe_fwd"].with_(name="scored", T=300, d=256, n_experts=16, top_k=4, inter=128,
                                           n_vdev=4, renorm=True, prof_tokens=2048)
    case = make_case(cfg, device="cuda:0")
    bias = (np.random.default_rng(2).normal(size=16) * 0.1).astype(np.float32)
    kw = dict(n_groups=4, keep=2, best=2, by_vdev=True, scale=1.5, sigmoid=sigmoid)
    score = occ.occult_score_t(score=occ.SCORE_SIGMOID if sigmoid else occ.SCORE_SOFTMAX, n_groups=4,
                               keep_groups=2, group_best=2, group_kind=occ.GROUP_VDEV, scale=1.5)
    moe = occ.OccultMoE(occ.desc_for(cfg), case.weights, torch.as_tensor(case.placement), score=score,
                        bias=torch.as_tensor(bias), merge=merge)
    y = moe.forward(case.logits.cuda(), case.x)
    torch.cuda.synchronize()
    assert occ.device_error() == 0
    e2v = moe.expert_to_vdev.cpu().numpy()
    ids, gates, _ = scored.route(case.logits.numpy(), 4, e2v, bias=bias, **kw)
    assert (moe.ids.cpu().numpy() == ids).all()
    f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    ref = oexpert.layer_output(f(case.x), ids, gates, {k: f(v) for k, v in case.weights.items()})
    assert_close_layer(y.float().cpu().numpy(), ref, cfg.dtype)


def reference(model, r, labels, teacher):
    """fp64 autograd of the chain from the residual stream to the total loss."""
    block, head = model.block, model.head
    ds, moe, o = block.desc, block.moe, head.opt
    p = {n: t.detach().double().requires_grad_() for n, t, _ in model.parameters()}
    r = r.double().requires_grad_()
    norm = lambda v: v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    x = norm(r) * p["w_pre"]
    logits = x @ p["w_router"].T
    ids = moe.ids.long()
    gates = logits.sigmoid().gather(1, ids)
    gates = moe.score.scale * gates / gates.sum(1, keepdim=True)
    I = ds.inter
    y = torch.zeros_like(x)
    for e in range(ds.n_experts):
        rows, slot = (ids == e).nonzero(as_tuple=True)
        w1, w2 = p["w1"].view(ds.n_experts, 2 * I, ds.d)[e], p["w2"].view(ds.n_experts, ds.d, I)[e]
        G, U = x[rows] @ w1[:I].T, x[rows] @ w1[I:].T
        y = y.index_add(0, rows, gates[rows, slot][:, None] * ((torch.nn.functional.silu(G) * U) @ w2.T))
    out = r + p["gate"] * (norm(y) * p["w_post"])
    aux = block.bal_opt.coef_z * logits.logsumexp(1).square().mean()
    z = (norm(out) * p["w_norm"]) @ p["w_head"].T
    lse = z.logsumexp(1)
    on = labels >= 0
    ce = (lse - z.gather(1, labels.clamp(min=0).long()[:, None])[:, 0])[on].mean()
    total = o.coef * ce
    every = on
    if teacher is not None:
        ti, tl = teacher
        kd_on = ti[:, 0] >= 0
        every = on | kd_on
        q = (tl.double() / o.temperature).softmax(1)
        logp = (z / o.temperature).log_softmax(1).gather(1, ti.clamp(min=0).long())
        total = total + o.coef_kd * o.temperature ** 2 * ((q * (q.log() - logp)).sum(1))[kd_on].mean()
    total = total + o.coef_z * lse[every].square().mean()
    (total + aux).backward()
    return total.detach(), r.grad, {n: t.grad for n, t in p.items()}


@pytest.mark.parametrize("distill", [False, True])
def test_gradients_of_the_whole_chain(occ, distill):
    from train_model import Model, batch
    cfg = config()
    K = 6 if distill else 0
    model = Model(cfg, VOCAB, topk=K, coef=0.6, coef_kd=0.4 if distill else 0.0, coef_z=1e-2, temperature=2.0)
    block = model.block
    block.moe.w["w1"].mul_(4)      # activations of order one in a layer this narrow
    block.moe.w["w2"].mul_(4)
    g = torch.Generator(device="cuda").manual_seed(3)
    block.moe.bias.copy_(0.1 * torch.randn(8, generator=g, device="cuda"))
    pairs, labels, teacher = batch(cfg, VOCAB, 1, K)
    labels[::7] = -100
    if distill:
        teacher[0][3::5, 0] = -1
    losses = model.gradients(pairs, labels, teacher)
    total, dr, grads = reference(model, model.stream(pairs), labels, teacher)
    torch.cuda.synchronize()
    assert occ.device_error() == 0
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert abs(float(losses[0]) / float(total) - 1) < REL
    assert rel(block.dr, dr) < REL
    for name, _, grad in model.parameters():
        assert rel(grad.view_as(grads[name]), grads[name]) < REL, name
    # the loss alone, on the same stream
    again = model.head.loss(block.r_out, labels, teacher)
    assert abs(float(again[0]) / float(total) - 1) < REL


def test_update_and_bias_move_what_they_are_given(occ):
    """A step of the optimizer over block and head changes every weight; the bias follows
    the last forward's counts."""
    from train_model import Model, batch
    cfg = config()
    model = Model(cfg, VOCAB)
    opt = model.optimizer(lr=1e-2)
    pairs, labels, _ = batch(cfg, VOCAB, 0, 0)
    model.gradients(pairs, labels)
    before = [p.clone() for _, p, _ in model.parameters()]
    opt.step()
    for (name, p, _), old in zip(model.parameters(), before):
        assert (p != old).any(), name
    counts = model.block.counts.cpu().numpy()
    model.block.bias_step()
    want = scored.bias_step(np.zeros(8), counts, 1e-3)
    np.testing.assert_allclose(model.block.moe.bias.cpu().numpy(), want, rtol=1e-6)


def test_step_replays_from_a_graph(occ):
    """Block, head and both backwards captured once and replayed on another batch."""
    from train_model import Model, batch
    cfg = config()
    model = Model(cfg, VOCAB, topk=4, coef=0.5, coef_kd=0.5, temperature=2.0)
    batches = [batch(cfg, VOCAB, i, 4) for i in (0, 1)]
    pairs, labels = batches[0][0].clone(), batches[0][1].clone()
    teacher = tuple(t.clone() for t in batches[0][2])

    def fill(b):
        pairs.copy_(b[0])
        labels.copy_(b[1])
        for t, v in zip(teacher, b[2]):
            t.copy_(v)

    want = []
    for b in batches:
        fill(b)
        losses = model.gradients(pairs, labels, teacher).clone()
        want.append((losses, model.head.dw.clone(), model.head.dx.clone()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        model.gradients(pairs, labels, teacher)
    for i in (0, 1, 0):
        fill(batches[i])
        g.replay()
        torch.cuda.synchronize()
        # (the layer's merge adds in no fixed order: equal up to fp32 roundings that bf16
        # activations pass on now and then)
        for a, b in zip((model.head.losses, model.head.dw, model.head.dx), want[i]):
            assert float((a - b).norm() / b.norm()) < REL
    assert occ.device_error() == 0


@pytest.mark.parametrize("args", [["--steps", "3"], ["--steps", "3", "--distill"]])
def test_example_runs(occ, args):
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "train_model.py"), *args],
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.count("step ") == 3 and "loads of the experts" in out.stdout


def test_refusals(occ):
    cfg = config()
    w = synth.expert_weights(cfg, device="cuda")
    placement = torch.arange(8, dtype=torch.int32).view(4, 2)
    with pytest.raises(ValueError, match="scored router"):
        occ.OccultMoE(occ.desc_for(cfg), w, placement, bias=torch.zeros(8))
    with pytest.raises(ValueError, match="route_mode"):
        occ.OccultMoE(occ.desc_for(cfg.with_(route_mode="score_pruned")), w, placement,
                      score=occ.occult_score_t())
    block = occ.OccultBlock(occ.desc_for(cfg), w, placement, torch.zeros(8, 128), score=occ.occult_score_t())
    with pytest.raises(RuntimeError, match="no bias"):
        block.bias_step()
    with pytest.raises(ValueError, match="w_head"):
        occ.OccultHead(occ.desc_for(cfg), torch.zeros(10, 64))
