"""Trains a one-block language model on a synthetic language and prints its losses.

    python examples/train_model.py [--steps 60] [--distill]

The next token of the language is a fixed random function of the two tokens before it.
The model: a fixed random embedding of those two, one MoE block whose router scores by
sigmoids under a bias that evens out the loads, and the output head.  With --distill the
head also learns from a teacher's top logits (here the language's own: most of the mass
on the next token, the rest on seven others).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_top_route_gb300 as occ  # noqa: E402
import synth  # noqa: E402


class Model:
    """Block and head over the residual stream of a batch of T token pairs."""

    def __init__(self, cfg, vocab, topk=0, seed=0, device="cuda", **head):
        g = torch.Generator(device=device).manual_seed(seed)
        placement = torch.arange(cfg.n_experts, dtype=torch.int32).view(cfg.n_vdev, -1)
        randn = lambda *n: torch.randn(*n, generator=g, device=device)  # noqa: E731
        score = occ.occult_score_t(n_groups=cfg.n_vdev, keep_groups=max(1, cfg.n_vdev // 2), group_best=2,
                                   group_kind=occ.GROUP_VDEV, scale=1.0, bias_rate=1e-3)
        self.block = occ.OccultBlock(occ.desc_for(cfg), synth.expert_weights(cfg, device=device), placement,
                                     0.05 * randn(cfg.n_experts, cfg.d), device=device,
                                     gate=torch.full((cfg.d,), 0.5), balance=(0.0, 0.0, 0.001),
                                     score=score, bias=torch.zeros(cfg.n_experts))
        self.head = occ.OccultHead(occ.desc_for(cfg), (cfg.d ** -0.5 * randn(vocab, cfg.d)).bfloat16(),
                                   device=device, topk=topk, **head)
        self.embed = randn(2, vocab, cfg.d).bfloat16()

    def parameters(self):
        return self.block.parameters() + self.head.parameters()

    def optimizer(self, **kw):
        ps = self.parameters()
        return occ.OccultAdamW([p for _, p, _ in ps], [g for _, _, g in ps], **kw)

    def stream(self, pairs):
        """The residual stream of token pairs [T, 2]."""
        return self.embed[0][pairs[:, 0]] + self.embed[1][pairs[:, 1]]

    def gradients(self, pairs, labels=None, teacher=None):
        """Losses [4]; every weight's gradient is left in its buffer."""
        r = self.block.forward(self.stream(pairs))
        losses, dr = self.head.step(r, labels, teacher)
        self.block.backward(dr)
        return losses


def batch(cfg, vocab, step, topk, device="cuda"):
    """(pairs, labels, teacher) of a step."""
    g = torch.Generator(device=device).manual_seed(100 + step)
    rule = torch.Generator(device=device).manual_seed(1)
    table = torch.randint(0, vocab, (vocab,), generator=rule, device=device)
    pairs = torch.randint(0, 64, (cfg.T, 2), generator=g, device=device)   # of the 64 commonest
    labels = table[(pairs[:, 0] * 64 + pairs[:, 1]) % vocab].int()
    teacher = None
    if topk:
        others = torch.randint(0, vocab, (cfg.T, topk - 1), generator=g, device=device).int()
        logits = torch.full((cfg.T, topk), 0.0, device=device)
        logits[:, 0] = 5.0
        teacher = torch.cat([labels[:, None], others], dim=1).contiguous(), logits
    return pairs, labels, teacher


def train(model, cfg, vocab, steps, topk=0, lr=2e-3):
    """[T losses {total, cross entropy, distillation, z}] of every step."""
    opt = model.optimizer(lr=lr, weight_decay=0.01)
    history = []
    for i in range(steps):
        pairs, labels, teacher = batch(cfg, vocab, i, topk)
        history.append(model.gradients(pairs, labels, teacher).clone())
        model.block.bias_step()
        opt.step()
    return torch.stack(history)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--distill", action="store_true")
    a = ap.parse_args()
    cfg = synth.CONFIGS["olmoe_train"].with_(name="example", T=4096, d=512, inter=256, n_experts=16,
                                             top_k=4, n_vdev=4, renorm=True)
    vocab, topk = 8192, 8 if a.distill else 0
    model = Model(cfg, vocab, topk=topk, coef=0.5 if a.distill else 1.0,
                  coef_kd=0.5 if a.distill else 0.0, coef_z=1e-4, temperature=2.0)
    h = train(model, cfg, vocab, a.steps, topk=topk).cpu()
    for i in sorted(set(range(0, a.steps, max(1, a.steps // 10))) | {a.steps - 1}):
        print(f"step {i:4d}  total {h[i, 0]:.4f}  cross entropy {h[i, 1]:.4f}  distillation {h[i, 2]:.4f}")
    print("loads of the experts:", model.block.counts[0].tolist())
    code = occ.device_error()
    if code:
        raise SystemExit(f"device error {code}: {occ.strerror(code)}")


if __name__ == "__main__":
    main()
