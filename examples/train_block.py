"""Trains one MoE block on a synthetic regression and prints its losses.

    python examples/train_block.py [--steps 60] [--state-bits 8] [--no-masters]

The block (norm, router, MoE layer, norm, gate, residual) learns to add a fixed
random nonlinear function of its input to the residual stream; the balance loss
keeps the experts' loads even meanwhile.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_top_route_gb300 as occ  # noqa: E402
import synth  # noqa: E402


def make_block(cfg, seed=0, device="cuda"):
    """A block of the configuration with small random weights."""
    g = torch.Generator(device=device).manual_seed(seed)
    placement = torch.arange(cfg.n_experts, dtype=torch.int32).view(cfg.n_vdev, -1)
    w_router = 0.05 * torch.randn(cfg.n_experts, cfg.d, generator=g, device=device)
    return occ.OccultBlock(occ.desc_for(cfg), synth.expert_weights(cfg, device=device), placement,
                           w_router, device=device, gate=torch.full((cfg.d,), 0.5),
                           balance=(0.02, 0.01, 0.001))


def train(block, cfg, steps, lr=2e-3, state_bits=32, masters=True, seed=1, device="cuda"):
    """[(regression loss, expert term of the balance loss)] of every step, on the GPU."""
    g = torch.Generator(device=device).manual_seed(seed)
    r = torch.randn(cfg.T, cfg.d, generator=g, device=device).bfloat16()
    teacher = torch.randn(cfg.d, cfg.d, generator=g, device=device) / cfg.d ** 0.5
    target = r.float() + torch.tanh(r.float() @ teacher)
    opt = block.optimizer(lr=lr, weight_decay=0.01, state_bits=state_bits, masters=masters)
    history = []
    for _ in range(steps):
        diff = block.forward(r).float() - target
        history.append(torch.stack([diff.square().mean(), block.losses[1]]))
        # the sum over channels of the mean over tokens: gradients of a usual size
        block.backward((2.0 / cfg.T * diff).to(r.dtype))
        opt.step()
    return torch.stack(history)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    ap.add_argument("--no-masters", action="store_true")
    a = ap.parse_args()
    cfg = synth.CONFIGS["olmoe_train"].with_(name="example", T=4096, d=512, inter=256,
                                             n_experts=16, top_k=4, n_vdev=4)
    block = make_block(cfg)
    h = train(block, cfg, a.steps, state_bits=a.state_bits, masters=not a.no_masters).cpu()
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  regression {h[i, 0]:.4f}  balance {h[i, 1]:.4f}")
    print(f"last       regression {h[-1, 0]:.4f}  balance {h[-1, 1]:.4f}")
    print("loads of the experts:", block.counts[0].tolist())
    code = occ.device_error()
    if code:
        raise SystemExit(f"device error {code}: {occ.strerror(code)}")


if __name__ == "__main__":
    main()
