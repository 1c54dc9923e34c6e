"""The output head's losses and gradients, in fp64, one token at a time.

z = x w^T.  Cross entropy over the tokens whose label lies in the vocabulary,
distillation over those whose first teacher token does (tau^2 times the mean of
KL(q || softmax(z / tau)), q the softmax of the teacher's entries over tau), and the mean
square of log sum exp z over the tokens that either counts.  A teacher row whose logits
are all -inf counts as a token and adds nothing.
"""
from __future__ import annotations

import numpy as np


def _lse(z):
    m = z.max()
    return m + np.log(np.exp(z - m).sum())


def losses(x, w, labels=None, t_ids=None, t_logits=None, tau=1.0, coef=1.0, coef_kd=0.0,
           coef_z=0.0, dloss=1.0, grads=True):
    """dict of loss [4], lse [T], token_loss [T], dx [T, d], dw [V, d]."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    T, V = len(x), len(w)
    inside = lambda v: 0 <= v < V  # noqa: E731
    ce_on = [labels is not None and inside(labels[t]) for t in range(T)]
    kd_on = [t_ids is not None and inside(t_ids[t][0]) for t in range(T)]
    n_ce, n_kd = max(1, sum(ce_on)), max(1, sum(kd_on))
    n = max(1, sum(a or b for a, b in zip(ce_on, kd_on)))
    lse, token = np.zeros(T), np.zeros(T)
    dx, dw = np.zeros_like(x), np.zeros_like(w)
    ce = kd = zz = 0.0
    for t in range(T):
        if not (ce_on[t] or kd_on[t]):
            continue
        z = w @ x[t]
        lse[t] = _lse(z)
        zz += lse[t] ** 2 / n
        dz = coef_z / n * 2 * lse[t] * np.exp(z - lse[t])
        if ce_on[t]:
            token[t] = lse[t] - z[labels[t]]
            ce += token[t] / n_ce
            dz += coef / n_ce * np.exp(z - lse[t])
            dz[labels[t]] -= coef / n_ce
        if kd_on[t]:
            on = [k for k in range(len(t_ids[t])) if inside(t_ids[t][k])]
            tl = np.asarray([t_logits[t][k] for k in on], dtype=np.float64) / tau
            if tl.max() > -np.inf:
                q = np.exp(tl - _lse(tl))
                logp = z / tau - _lse(z / tau)
                for k, qk in zip(on, q):
                    if qk > 0:
                        kd += tau * tau / n_kd * qk * (np.log(qk) - logp[t_ids[t][k]])
                    dz[t_ids[t][k]] -= coef_kd * tau / n_kd * qk
                dz += coef_kd * tau / n_kd * np.exp(logp)
        if grads:
            dx[t] = dloss * (dz @ w)
            dw += dloss * np.outer(dz, x[t])
    total = coef * ce + coef_kd * kd + coef_z * zz
    return dict(loss=np.array([total, ce, kd, zz]), lse=lse, token_loss=token, dx=dx, dw=dw)
