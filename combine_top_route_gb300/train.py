"""One MoE block in training: the layer between its norms, its losses and its update;
and the head that ends a model.

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

``OccultHead`` is the last norm and the loss over a vocabulary: labels, a teacher's top
logits, or both, forward and backward in one call.
``OccultAdamW`` is the update on its own, for any tensors with fp32 gradients.
"""
from __future__ import annotations

from typing import Dict, Optional, Sequence

import torch

from . import (GATE_CHANNEL, GATE_NONE, OCCULT_BF16, OCCULT_F32, STATE_BLOCK, STATE_M, STATE_V,
               WS_BLOCK_NORM_BWD, adamw_table, balance_groups, balance_workspace_size,
               occult_adamw, occult_adamw_read, occult_adamw_t, occult_balance_grad,
               occult_balance_loss, occult_balance_t, occult_block_norm, occult_block_norm_bwd,
               head_workspace_size, occult_desc_t, occult_head_loss, occult_head_step,
               occult_head_t, occult_norm_t, occult_route_bias_step, occult_score_t,
               workspace_size)
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
                 balance=(0.01, 0.0, 0.001), group_len: int = 0, sim_table=None,
                 score: Optional[occult_score_t] = None, bias: Optional[torch.Tensor] = None):
        """``weights``: w1 and w2 as OccultMoE takes them (bf16 ones on the device are
        used where they are, so that an optimizer's steps change the caller's tensors;
        the other weights are copied); ``w_router`` fp32 [Ne, d];
        ``gate`` fp32 [d] or None; ``balance``: the weights of the expert, device and z
        terms, which are made from softmax(logits) whatever the router's scores are: beside a
        router of sigmoids the expert and device terms pull at probabilities that choose
        nothing, and a bias evens the loads out instead (weights 0, 0);
        ``group_len``: tokens of a sequence for them (0: the batch); ``score`` and
        ``bias``: the scored router's, as OccultMoE takes them."""
        if desc.dtype != OCCULT_BF16 or desc.n_shared:
            raise ValueError("OccultBlock trains bf16 layers without shared experts")
        self.desc = desc
        self.moe = OccultMoE(desc, weights, placement, device=device, train=True,
                             sim_table=sim_table, score=score, bias=bias)
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
        self.counts = torch.zeros(G, Ne, dtype=torch.int32, device=dev)
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

    def bias_step(self, stream=None) -> None:
        """Moves the scored router's bias towards even loads, by the last forward's counts."""
        if self.moe.bias is None:
            raise RuntimeError("the block's router has no bias")
        occult_route_bias_step(self.desc, self.moe.score, self.counts, self.moe.bias, stream)

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


class OccultHead:
    """The end of a model: the last norm, the product with the vocabulary and its losses.

    Every row of the residual stream must be finite, those that no term counts as well: the
    norm's weight sums over all of them (a row that counts nowhere adds 0 times its norm).
    """

    def __init__(self, desc: occult_desc_t, w_head: torch.Tensor, device="cuda", eps: float = 1e-6,
                 res_dtype=torch.bfloat16, topk: int = 0, coef: float = 1.0, coef_kd: float = 0.0,
                 coef_z: float = 0.0, temperature: float = 1.0, piece: int = 0, train: bool = True):
        """``desc``: T, d and dtype are the head's; ``w_head`` [V, d] (in the layer type and on
        the device it is used where it is); ``topk``: teacher entries a token; the other
        options as in occult_head_t; ``train=False``: ``loss`` alone, without the gradients'
        buffers and the workspace of a step's logits."""
        dev, dt = torch.device(device), desc.torch_dtype
        T, d, V = desc.T, desc.d, w_head.shape[0]
        if tuple(w_head.shape) != (V, d):
            raise ValueError(f"w_head must be [V, {d}]")
        self.desc = desc
        self.opt = occult_head_t(vocab=V, topk=topk, coef=coef, coef_kd=coef_kd, coef_z=coef_z,
                                 temperature=temperature, piece=piece)
        self.norm_opt = occult_norm_t(eps, 1.0, GATE_NONE,
                                      OCCULT_BF16 if res_dtype == torch.bfloat16 else OCCULT_F32)
        e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
        self.w = w_head.to(dev, dt).contiguous()
        self.w_norm = torch.ones(d, dtype=dt, device=dev)
        self.x, self.rstd = e(T, d, dtype=dt), e(T)
        self.losses, self.lse, self.token_loss = e(4), e(T), e(T)
        self.train = train
        self.dx = self.dr = self.dw = self.dw_norm = self.norm_ws = None
        need = head_workspace_size(desc, self.opt, step=False)
        if train:
            self.dx, self.dr, self.dw, self.dw_norm = e(T, d), e(T, d, dtype=res_dtype), e(V, d), e(d)
            self.norm_ws = e(max(1, workspace_size(desc, WS_BLOCK_NORM_BWD)), dtype=torch.uint8)
            need = max(need, head_workspace_size(desc, self.opt, step=True))
        self.ws = e(max(1, need), dtype=torch.uint8)

    def _trains(self):
        if not self.train:
            raise RuntimeError("OccultHead was built without train=True")

    def parameters(self):
        """[(name, parameter, its fp32 gradient)], as OccultBlock.parameters."""
        self._trains()
        return [("w_head", self.w, self.dw), ("w_norm", self.w_norm, self.dw_norm)]

    def _norm(self, r):
        occult_block_norm(self.desc, self.norm_opt, r, w_pre=self.w_norm, x=self.x, rstd_pre=self.rstd)

    def _inputs(self, labels, teacher):
        ids, logits = (None, None) if teacher is None else teacher
        if labels is None:
            self.token_loss.zero_()
        return dict(labels=labels, teacher_ids=ids, teacher_logits=logits, lse=self.lse,
                    token_loss=None if labels is None else self.token_loss)

    def loss(self, r: torch.Tensor, labels: Optional[torch.Tensor] = None, teacher=None):
        """[4] {total, cross entropy, distillation, z} of the residual stream r, without a
        gradient; ``labels`` int32 [T], ``teacher`` (int32 [T, K] tokens, fp32 [T, K] logits).
        The tokens' own losses are left in ``token_loss`` (0 without labels), their log-sums in
        ``lse``."""
        self._norm(r)
        occult_head_loss(self.desc, self.opt, self.x, self.w, self.losses, self.ws,
                         **self._inputs(labels, teacher))
        return self.losses

    def step(self, r: torch.Tensor, labels: Optional[torch.Tensor] = None, teacher=None,
             dloss: Optional[torch.Tensor] = None):
        """(losses [4], gradient of r): as ``loss``, with the total's gradients (times the
        fp32 CUDA tensor ``dloss``); the weights' are left in their buffers."""
        self._trains()
        self._norm(r)
        occult_head_step(self.desc, self.opt, self.x, self.w, self.losses, self.ws, dx=self.dx,
                         dw=self.dw, dloss=dloss, **self._inputs(labels, teacher))
        occult_block_norm_bwd(self.desc, self.norm_opt, None, r, self.dr, self.norm_ws, dx=self.dx,
                              w_pre=self.w_norm, rstd_pre=self.rstd, dw_pre=self.dw_norm)
        return self.losses, self.dr
