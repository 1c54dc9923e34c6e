"""The block in training: its gradients against fp64 autograd of the same formulas,
its updates, and that training it lowers the loss in every state format.

Tolerance of the gradients (2-norm of the difference over that of the gradient):
activations pass some ten roundings to bf16 of relative size 2^-9 (uniform: 2^-9 /
sqrt(3) each in the 2-norm), the saved pre-activations among them whose error enters
twice; independent, that is 2^-9 sqrt(20 / 3) < 0.6 %.  1.5 % leaves room for the
amplification by the norms and the router's small differences of gates.
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
    return occ


def config(T=384, renorm=False):
    return synth.CONFIGS["olmoe_train"].with_(name="block", T=T, d=128, inter=64, n_experts=8,
                                              top_k=2, n_vdev=4, renorm=renorm)


def reference(block, r, dr_out, mask):
    """fp64 autograd of the block's formulas with the routing as the block chose it."""
    ds, moe = block.desc, block.moe
    p = {n: t.detach().double().requires_grad_() for n, t, _ in block.parameters()}
    r = r.double().requires_grad_()
    eps = block.pre_opt.eps

    def norm(v):
        return v * (v.square().mean(1, keepdim=True) + eps).rsqrt()

    x = norm(r) * p["w_pre"]
    logits = x @ p["w_router"].T
    prob = logits.softmax(1)
    ids = moe.ids.long()
    gates = prob.gather(1, ids)
    if ds.renorm:
        gates = gates / gates.sum(1, keepdim=True)
    I = ds.inter
    y = torch.zeros_like(x)
    for e in range(ds.n_experts):
        rows, slot = (ids == e).nonzero(as_tuple=True)
        w1, w2 = p["w1"].view(ds.n_experts, 2 * I, ds.d)[e], p["w2"].view(ds.n_experts, ds.d, I)[e]
        G, U = x[rows] @ w1[:I].T, x[rows] @ w1[I:].T
        y = y.index_add(0, rows, gates[rows, slot][:, None] * ((torch.nn.functional.silu(G) * U) @ w2.T))
    out = block.post_opt.res_scale * r + p["gate"] * (norm(y) * p["w_post"])
    on = torch.ones(ds.T, device=r.device, dtype=torch.float64) if mask is None else mask.double()
    N = on.sum()
    f = torch.zeros(ds.n_experts, dtype=torch.float64, device=r.device)
    f.index_add_(0, ids.reshape(-1), on[:, None].expand_as(ids).reshape(-1))
    f = f * ds.n_experts / (ds.top_k * N)
    P = (prob * on[:, None]).sum(0) / N
    onehot = torch.nn.functional.one_hot(moe.expert_to_vdev.long(), ds.n_vdev).double()
    dev = ((f @ onehot) / onehot.sum(0) * (P @ onehot)).sum()
    z = (logits.logsumexp(1).square() * on).sum() / N
    b = block.bal_opt
    aux = b.coef * (f * P).sum() + b.coef_dev * dev + b.coef_z * z
    ((out * dr_out.double()).sum() + aux).backward()
    return out.detach(), aux.detach(), r.grad, {n: t.grad for n, t in p.items()}


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_gradients_of_the_whole_block(occ, masked, renorm):
    from train_block import make_block
    cfg = config(renorm=renorm)
    block = make_block(cfg)
    block.moe.w["w1"].mul_(4)      # activations of order one in a layer this narrow
    block.moe.w["w2"].mul_(4)
    block.bal_opt.coef, block.bal_opt.coef_dev, block.bal_opt.coef_z = 20.0, 10.0, 2.0
    g = torch.Generator(device="cuda").manual_seed(3)
    r = torch.randn(cfg.T, cfg.d, generator=g, device="cuda").bfloat16()
    up = torch.randn(cfg.T, cfg.d, generator=g, device="cuda").bfloat16()
    mask = (torch.rand(cfg.T, generator=g, device="cuda") < 0.8).to(torch.uint8) if masked else None
    out = block.forward(r, mask)
    dr = block.backward(up)
    want_out, aux, want_dr, grads = reference(block, r, up, mask)
    torch.cuda.synchronize()
    assert occ.device_error() == 0

    def rel(a, b):
        return float((a.double() - b).norm() / b.norm())

    assert rel(out, want_out) < REL
    assert abs(float(block.losses[0]) / float(aux) - 1) < REL
    assert rel(dr, want_dr) < REL
    for name, p, grad in block.parameters():
        assert rel(grad.view_as(grads[name]), grads[name]) < REL, name


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("masters", [True, False])
def test_training_lowers_the_loss(occ, state_bits, masters):
    from train_block import make_block, train
    cfg = config(T=1024)
    block = make_block(cfg)
    h = train(block, cfg, 80, state_bits=state_bits, masters=masters).cpu().numpy()
    assert np.isfinite(h).all()
    assert h[-5:, 0].mean() < 0.75 * h[0, 0]
    assert block.counts.sum().item() == cfg.T * cfg.top_k
    assert occ.device_error() == 0


def test_optimizer_updates_every_parameter(occ):
    from train_block import make_block
    cfg = config()
    block = make_block(cfg)
    opt = block.optimizer(lr=1e-2, state_bits=8)
    before = [p.clone() for _, p, _ in block.parameters()]
    r = torch.randn(cfg.T, cfg.d, device="cuda").bfloat16()
    block.forward(r)
    block.backward(torch.ones_like(r))
    opt.step(grad_scale=torch.ones(1, device="cuda"))
    for (name, p, g), b in zip(block.parameters(), before):
        # the first step moves every weight with a gradient by the rate against its sign
        live = g.view(-1).abs() > 1e-6
        moved = (p.float() - b.float()).view(-1)[live]
        assert (moved * g.view(-1)[live] <= 0).float().mean() > 0.99, name
        m, v = opt.moments(0)
        assert m.dtype == torch.float32 and (v >= 0).all()
    with pytest.raises(ValueError):
        opt.step(grad_scale=torch.ones(1))
    with pytest.raises(ValueError):
        occ.OccultAdamW([before[0]], [], lr=1e-3)
    with pytest.raises(ValueError):
        occ.OccultAdamW([before[0]], [before[0].float()], lr=1e-3, state_bits=16)


@pytest.mark.parametrize("masked", [False, True])
def test_loads_under_pruning_are_those_the_layer_carries(occ, masked):
    """Similarity-based pruning puts other experts in the place of some that the router
    chose: counts, losses and the losses' gradient are of the experts that run.  (Counts
    exact; sums of positive terms within 1100 units of fp32, 7e-5, of themselves, and a
    gradient within 1e-4 of its largest element, as no term of it is larger.)"""
    from oracle import balance as obal
    cfg = config().with_(route_mode="similarity_pruned", limit_devices=1, n_clusters=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    placement = torch.arange(cfg.n_experts, dtype=torch.int32).view(cfg.n_vdev, -1)
    block = occ.OccultBlock(occ.desc_for(cfg), synth.expert_weights(cfg, device="cuda"), placement,
                            0.3 * torch.randn(cfg.n_experts, cfg.d, generator=g, device="cuda"),
                            balance=(0.3, 0.2, 0.1), group_len=100,
                            sim_table=synth.random_similarity_table(cfg))
    r = torch.randn(cfg.T, cfg.d, generator=g, device="cuda").bfloat16()
    mask = (torch.rand(cfg.T, generator=g, device="cuda") < 0.8).to(torch.uint8) if masked else None
    block.forward(r, mask)
    block.backward(torch.zeros_like(r))      # what is left in dlogits is the losses' gradient
    torch.cuda.synchronize()
    assert not torch.equal(block.moe.ids, block.moe.routed)
    host = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    loss, counts, grad = obal.loss_and_grad(
        host(block.logits), host(block.moe.ids), host(block.moe.expert_to_vdev), cfg.n_vdev, 100,
        host(mask), coef=0.3, coef_dev=0.2, coef_z=0.1)
    assert (host(block.counts) == counts).all()
    np.testing.assert_allclose(host(block.losses), loss, rtol=1e-4)
    assert np.abs(host(block.moe.dlogits) - grad).max() <= 1e-4 * np.abs(grad).max()


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("raw", [False, True])
def test_moments_are_read_behind_the_steps_of_their_stream(occ, state_bits, raw):
    """Steps and read-out on a side stream that still has other work before them."""
    g = torch.Generator(device="cuda").manual_seed(2)
    p = torch.randn(70000, generator=g, device="cuda").bfloat16()
    grad = torch.randn(70000, generator=g, device="cuda")
    opt = occ.OccultAdamW([p], [grad], lr=1e-3, state_bits=state_bits)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)        # some 30 ms
    on = s.cuda_stream if raw else s
    opt.step(stream=on)
    m, v = opt.moments(0, stream=on)
    s.synchronize()
    want_m, want_v = opt.moments(0)
    torch.cuda.synchronize()
    assert torch.equal(m, want_m) and torch.equal(v, want_v)
    # (and they are a first step's: (1 - beta1) g within a code's unit)
    assert ((m - 0.1 * grad).abs() <= 0.13 * (0.1 * grad).abs() + 1e-4).all()


@pytest.mark.parametrize("raw", [False, True])
def test_a_factor_of_the_gradients_outlives_its_step(occ, raw):
    """Factors dropped by the host while a busy side stream has yet to read them: their
    memory goes to nothing that the current stream writes meanwhile."""
    p = torch.zeros(4096, device="cuda")
    grad = torch.ones(4096, device="cuda")
    opt = occ.OccultAdamW([p], [grad], lr=1e-3)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)        # some 30 ms
    m = 0.0
    for i in range(8):
        factor = torch.empty(1, device="cuda")
        with torch.cuda.stream(s):
            factor.fill_(2.0 ** i)           # written and read behind the other work
        opt.step(grad_scale=factor, stream=s.cuda_stream if raw else s)
        m = 0.9 * m + 0.1 * 2.0 ** i
        del factor
    torch.zeros(64, 1, device="cuda")
    keep = [torch.zeros(1, device="cuda") for _ in range(64)]
    s.synchronize()
    assert len(keep) == 64
    got = opt.states[0]["m"]
    assert ((got - m).abs() <= 1e-6 * m).all()


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("masters", [True, False])
def test_first_step_of_every_parameter(occ, state_bits, masters):
    """The first step from zero states: w (1 - lr wd) - lr g / (|g| + eps), m = (1 - b1) g and
    v = (1 - b2) g^2, for each parameter.  Tolerances: fp32 arithmetic (2^-18 of the terms);
    a bf16 parameter is its master's nearest value, or by a draw within a whole unit (2^-7);
    8-bit codes a unit of their binade (1/8 of m, 1/16 of the root of v) and, below a
    block's sixteen binades, what its largest value leaves (2^-15 of it, twice that where
    a rounding up moves the binades)."""
    from train_block import make_block
    cfg = config()
    block = make_block(cfg)
    lr, wd, eps = 1e-2, 0.1, 1e-8
    opt = block.optimizer(lr=lr, weight_decay=wd, eps=eps, state_bits=state_bits, masters=masters)
    g = torch.Generator(device="cuda").manual_seed(7)
    block.forward(torch.randn(cfg.T, cfg.d, generator=g, device="cuda").bfloat16())
    block.backward(torch.randn(cfg.T, cfg.d, generator=g, device="cuda").bfloat16())
    before = [p.detach().double().view(-1) for _, p, _ in block.parameters()]
    opt.step()

    def block_top(x):
        pad = torch.nn.functional.pad(x.abs(), (0, -len(x) % 256))
        return pad.view(-1, 256).amax(1).repeat_interleave(256)[:len(x)]

    for i, (name, p, grad) in enumerate(block.parameters()):
        dw = grad.double().view(-1)
        assert float((dw.abs() > 1e-7).float().mean()) > 0.9, name
        want = before[i] * (1 - lr * wd) - lr * dw / (dw.abs() + eps)
        tol = 2.0 ** -18 * (before[i].abs() + lr)
        got = p.view(-1)
        if p.dtype == torch.bfloat16 and masters:
            master = opt.states[i]["master"].view(-1)
            assert torch.equal(got, master.to(torch.bfloat16)), name
            got = master
        elif p.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -7 * want.abs()
        assert ((got.double() - want).abs() <= tol).all(), name
        m, v = (t.double() for t in opt.moments(i))
        for x, w, part in ((m, 0.1 * dw, 8), (v.sqrt(), 0.05 ** 0.5 * dw.abs(), 16)):
            err = 2.0 ** -18 * w.abs()
            if state_bits == 8:
                err = w.abs() / part * 1.001 + 2.0 ** -14 * block_top(w)
            assert ((x - w).abs() <= err + 1e-30).all(), (name, part)
