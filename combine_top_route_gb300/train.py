"""One MoE block in training: the layer between its norms, its losses and its update.

``OccultBlock`` runs a block r -> r' of a residual stream as a training step needs
it, every step but the router's three small matrix products in the library's
kernels:

    forward   x = norm(r) w_pre;  logits = x W_r^T;  y = layer(logits, x)
              auxiliary losses of the router (per-expert counts beside them)
              r' = res_scale r + gate norm(y) w_post
    backward  from the gradient of r' through the second norm, the layer, the
              router (the auxiliary losses' gradient added to the gates') and the
              first norm to the gradient of r and of every weight
    step      AdamW over all of the block's weights, up to 256 tensors a launch

``OccultAdamW`` is that update on its own, for any tensors with fp32 gradients.
"""
from __future__ import annotations

from typing import Dict, Optional, Sequence

import torch

from . import (GATE_CHANNEL, GATE_NONE, OCCULT_BF16, OCCULT_F32, STATE_BLOCK, STATE_M, STATE_V,
               WS_BLOCK_NORM_BWD, adamw_table, balance_groups, balance_workspace_size,
               occult_adamw, occult_adamw_read, occult_adamw_t, occult_balance_grad,
               occult_balance_loss, occult_balance_t, occult_block_norm, occult_block_norm_bwd,
               occult_desc_t, occult_norm_t, workspace_size)
from .pipeline import OccultMoE


def _torch_stream(stream):
    """torch's object for a stream given as one, as a handle, or not at all (None)."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)))


class OccultAdamW:
    """AdamW over tensors of one device, its states in fp32 or in 8 bits.

    ``params``: contiguous bf16 or fp32 tensors, updated in place; ``grads``: the
    fp32 buffers their gradients are written to before every ``step``.  ``masters``:
    keep an fp32 copy of every bf16 parameter (otherwise its update is rounded up
    or down by a draw).  The step's number and rate are the host's: ``step`` is called
    every time, not replayed from a CUDA graph, which would repeat the one captured.
    """

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], lr: float,
                 betas=(0.9, 0.95), eps: float = 1e-8, weight_decay: float = 0.1,
                 state_bits: int = 32, masters: bool = True, seed: int = 0):
        if len(params) != len(grads):
            raise ValueError("as many gradients as parameters are needed")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        self.params, self.grads = list(params), list(grads)
        st = torch.uint8 if state_bits == 8 else torch.float32
        self.states, first = [], 0
        for p, g in zip(self.params, self.grads):
            n = p.numel()
            blocks = -(-n // STATE_BLOCK)
            z = lambda k, dt: torch.zeros(k, dtype=dt, device=p.device)  # noqa: E731
            rec = dict(param=p, grad=g, m=z(n, st), v=z(n, st), first=first)
            if state_bits == 8:
                rec.update(m_exp=z(blocks, torch.uint8), v_exp=z(blocks, torch.uint8))
            if masters and p.dtype == torch.bfloat16:
                rec["master"] = p.float()
            self.states.append(rec)
            first += blocks * STATE_BLOCK
        self.table = adamw_table(self.states)
        self.opt = occult_adamw_t(lr=lr, beta1=betas[0], beta2=betas[1], eps=eps,
                                  weight_decay=weight_decay, step=0, state_bits=state_bits,
                                  seed=seed)
        self._scale = None

    def step(self, grad_scale: Optional[torch.Tensor] = None, lr: Optional[float] = None,
             stream=None) -> None:
        """One update; ``grad_scale``: a fp32 CUDA tensor [1] that multiplies the gradients."""
        if grad_scale is not None and (grad_scale.dtype != torch.float32
                                       or not grad_scale.is_cuda or grad_scale.numel() < 1):
            raise ValueError("grad_scale must be a float32 CUDA tensor")
        opt, before = self.opt, (self.opt.grad_scale, self.opt.lr, self.opt.step)
        opt.grad_scale = None if grad_scale is None else grad_scale.data_ptr()
        if lr is not None:
            opt.lr = lr
        opt.step += 1
        try:
            occult_adamw(opt, self.table, stream)
        except Exception:
            opt.grad_scale, opt.lr, opt.step = before  # a refused step is none
            raise
        self._scale = grad_scale  # alive until the next step, on the device until this one ran
        if grad_scale is not None:
            grad_scale.record_stream(_torch_stream(stream) or torch.cuda.current_stream())

    def moments(self, i: int, stream=None):
        """(m, v) of parameter ``i`` in fp32, as its state holds them; all of it on
        ``stream``, behind the steps there."""
        s = self.states[i]
        with torch.cuda.stream(_torch_stream(stream)):
            if self.opt.state_bits == 32:
                return s["m"].clone(), s["v"].clone()
            out = [torch.empty(s["m"].numel(), dtype=torch.bfloat16, device=s["m"].device)
                   for _ in range(2)]
            occult_adamw_read(s["m"], s["m_exp"], STATE_M, out[0])
            occult_adamw_read(s["v"], s["v_exp"], STATE_V, out[1])
            return out[0].float(), out[1].float().square()


class OccultBlock:
    """A block of one MoE layer in training (bf16, without shared experts)."""

    def __init__(self, desc: occult_desc_t, weights: Dict[str, torch.Tensor],
                 placement: torch.Tensor, w_router: torch.Tensor, device="cuda",
                 eps: float = 1e-6, res_scale: float = 1.0, res_dtype=torch.bfloat16,
                 post_norm: bool = True, gate: Optional[torch.Tensor] = None,
                 balance=(0.01, 0.0, 0.001), group_len: int = 0, sim_table=None):
        """``weights``: w1 and w2 as OccultMoE takes them (bf16 ones on the device are
        used where they are, so that an optimizer's steps change the caller's tensors;
        the other weights are copied); ``w_router`` fp32 [Ne, d];
        ``gate`` fp32 [d] or None; ``balance``: the weights of the expert, device and z
        terms; ``group_len``: tokens of a sequence for them (0: the batch)."""
        if desc.dtype != OCCULT_BF16 or desc.n_shared:
            raise ValueError("OccultBlock trains bf16 layers without shared experts")
        self.desc = desc
        self.moe = OccultMoE(desc, weights, placement, device=device, train=True,
                             sim_table=sim_table)
        dev = self.moe.device
        T, d, Ne = desc.T, desc.d, desc.n_experts
        f32, bf = torch.float32, torch.bfloat16
        e = lambda *s, dtype=f32: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
        self.w_router = w_router.to(dev, f32).contiguous().clone()
        self.w_pre = torch.ones(d, dtype=bf, device=dev)
        self.w_post = torch.ones(d, dtype=bf, device=dev) if post_norm else None
        self.gate = None if gate is None else gate.to(dev, f32).contiguous().clone()
        kind = OCCULT_BF16 if res_dtype == bf else OCCULT_F32
        self.pre_opt = occult_norm_t(eps, 1.0, GATE_NONE, kind)
        self.post_opt = occult_norm_t(eps, res_scale,
                                      GATE_NONE if gate is None else GATE_CHANNEL, kind)
        self.bal_opt = occult_balance_t(*balance, group_len)
        self.r = self.mask = self.x32 = None
        self.x, self.logits = e(T, d, dtype=bf), e(T, Ne)
        self.r_out, self.dr = e(T, d, dtype=res_dtype), e(T, d, dtype=res_dtype)
        self.dr_mid, self.dy = e(T, d, dtype=res_dtype), e(T, d, dtype=bf)
        self.rstd_pre = e(T)
        self.rstd_post = e(T) if post_norm else None
        G = balance_groups(desc, self.bal_opt)
        self.counts = e(G, Ne, dtype=torch.int32)
        self.grad_w, self.losses = e(G * Ne + 1), e(4)
        self.bal_ws = e(max(1, balance_workspace_size(desc, self.bal_opt)), dtype=torch.uint8)
        self.norm_ws = e(max(1, workspace_size(desc, WS_BLOCK_NORM_BWD)), dtype=torch.uint8)
        self.dw_pre = e(d)
        self.dw_post = e(d) if post_norm else None
        self.dgate = e(d) if gate is not None else None
        self.dw_router = e(Ne, d)

    def parameters(self):
        """[(name, parameter, its fp32 gradient)], updated by ``backward``."""
        out = [("w1", self.moe.w["w1"], self.moe.dw1), ("w2", self.moe.w["w2"], self.moe.dw2),
               ("w_router", self.w_router, self.dw_router), ("w_pre", self.w_pre, self.dw_pre)]
        if self.w_post is not None:
            out.append(("w_post", self.w_post, self.dw_post))
        if self.gate is not None:
            out.append(("gate", self.gate, self.dgate))
        return out

    def optimizer(self, **kw) -> OccultAdamW:
        """An OccultAdamW over the block's parameters."""
        ps = self.parameters()
        return OccultAdamW([p for _, p, _ in ps], [g for _, _, g in ps], **kw)

    def forward(self, r: torch.Tensor, mask: Optional[torch.Tensor] = None) -> torch.Tensor:
        """r' [T, d] for the residual stream r; the auxiliary losses in ``self.losses``
        ({weighted total, expert, device, z}), the experts' loads in ``self.counts``.
        ``mask`` (uint8 [T]): tokens with 0 take no part in the losses.  Under pruning
        that puts other experts in the place of some the router chose, losses and loads
        are of the experts that run."""
        ds, moe = self.desc, self.moe
        self.r, self.mask = r, mask
        occult_block_norm(ds, self.pre_opt, r, w_pre=self.w_pre, x=self.x, rstd_pre=self.rstd_pre)
        self.x32 = self.x.float()
        torch.mm(self.x32, self.w_router.t(), out=self.logits)
        y = moe.forward(self.logits, self.x)
        occult_balance_loss(ds, self.bal_opt, self.logits, moe.ids, moe.expert_to_vdev,
                            self.counts, self.grad_w, self.losses, self.bal_ws, mask=mask)
        occult_block_norm(ds, self.post_opt, r, y=y, w_post=self.w_post, gate=self.gate,
                          r_out=self.r_out, rstd_post=self.rstd_post)
        return self.r_out

    def backward(self, dr_out: torch.Tensor) -> torch.Tensor:
        """The gradient of r for the gradient dr_out of r' (plus the auxiliary losses'
        total); the weights' gradients are left in their buffers."""
        ds, moe = self.desc, self.moe
        occult_block_norm_bwd(ds, self.post_opt, dr_out, None, self.dr_mid, self.norm_ws,
                              y=moe.y, w_post=self.w_post, gate=self.gate,
                              rstd_post=self.rstd_post, dy=self.dy, dw_post=self.dw_post,
                              dgate=self.dgate)
        dx = moe.backward(self.dy)[0]
        occult_balance_grad(ds, self.bal_opt, self.logits, self.grad_w, moe.dlogits,
                            mask=self.mask, accumulate=True)
        torch.mm(moe.dlogits.t(), self.x32, out=self.dw_router)
        dx.addmm_(moe.dlogits, self.w_router)
        occult_block_norm_bwd(ds, self.pre_opt, self.dr_mid, self.r, self.dr, self.norm_ws, dx=dx,
                              w_pre=self.w_pre, rstd_pre=self.rstd_pre, dw_pre=self.dw_pre)
        return self.dr
