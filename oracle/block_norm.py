"""RMS norms around a block with its gate and residual scale, in fp64.

For one token, with rms(v) = (mean(v^2) + eps)^(1/2):

    b  = w_post y / rms(y)          (b = y without w_post)
    r' = a r + gate b
    x  = w_pre r' / rms(r')

``gate`` is None, a vector [d] (channels) or a column [T, 1] (tokens).
"""
from __future__ import annotations

import numpy as np


def rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1) + eps)


def forward(r, y=None, w_post=None, gate=None, w_pre=None, eps=1e-6, res_scale=1.0):
    """dict of r_out, x, rstd_post, rstd_pre (those that exist)."""
    out = {}
    s = np.asarray(r, dtype=np.float64)
    if y is not None:
        b = np.asarray(y, dtype=np.float64)
        if w_post is not None:
            out["rstd_post"] = rstd(b, eps)
            b = b * out["rstd_post"][:, None] * w_post
        s = res_scale * s + (b if gate is None else gate * b)
        out["r_out"] = s
    if w_pre is not None:
        out["rstd_pre"] = rstd(s, eps)
        out["x"] = s * out["rstd_pre"][:, None] * w_pre
    return out


def norm_back(v, c, dn):
    """Gradient with respect to v of <dn, c v>, c = (mean(v^2) + eps)^(-1/2)."""
    n = v * c[:, None]
    return c[:, None] * (dn - n * (dn * n).mean(axis=1, keepdims=True))


def backward(dr_out, dx, r_out, y=None, w_post=None, gate=None, w_pre=None, rstd_post=None,
             rstd_pre=None, res_scale=1.0):
    """Gradients of sum(dr_out r') + sum(dx x), with the saved row factors given."""
    out = {}
    shape = (dr_out if dr_out is not None else dx).shape
    D = np.zeros(shape) if dr_out is None else np.asarray(dr_out, dtype=np.float64)
    if w_pre is not None:
        D = D + norm_back(r_out, rstd_pre, dx * w_pre)
        out["dw_pre"] = (dx * r_out * rstd_pre[:, None]).sum(axis=0)
    if y is None:
        out["dr"] = D
        return out
    out["dr"] = res_scale * D
    m = y if w_post is None else y * rstd_post[:, None]
    b = m if w_post is None else m * w_post
    u = D
    if gate is not None:
        out["dgate"] = (D * b).sum(axis=0 if np.ndim(gate) == 1 else 1)
        u = u * gate
    if w_post is not None:
        out["dw_post"] = (u * m).sum(axis=0)
        u = norm_back(y, rstd_post, u * w_post)
    out["dy"] = u
    return out
