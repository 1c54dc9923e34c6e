"""The router's auxiliary losses and their gradient, in fp64, one group at a time.

Over the unmasked tokens of a group (N_g of them): c_e slots that chose expert e,
f_e = Ne c_e / (k N_g), P_e the mean probability.  expert = mean over the groups
that have tokens of sum_e f_e P_e; device = the same mean of sum_d (mean of f over
d's experts) (sum of P over them); z = mean over all tokens of (log sum exp)^2.
"""
from __future__ import annotations

import numpy as np


def groups(n_tokens, group_len):
    L = group_len if group_len > 0 else max(1, n_tokens)
    return [range(a, min(n_tokens, a + L)) for a in range(0, max(1, n_tokens), L)]


def loss_and_grad(logits, ids, expert_to_vdev, n_vdev, group_len=0, mask=None, coef=0.0,
                  coef_dev=0.0, coef_z=0.0):
    """(loss [4], counts [G, Ne], dlogits [T, Ne]) of the total's gradient."""
    T, Ne = logits.shape
    k = ids.shape[1] if ids.ndim == 2 else 1
    parts = groups(T, group_len)
    keep = [[t for t in g if mask is None or mask[t]] for g in parts]
    A = max(1, sum(1 for g in keep if g))
    N = max(1, sum(len(g) for g in keep))
    counts = np.zeros((len(parts), Ne), dtype=np.int64)
    dlogits = np.zeros((T, Ne))
    expert = device = z2 = 0.0
    for gi, toks in enumerate(keep):
        if not toks:
            continue
        z = np.asarray(logits[toks], dtype=np.float64)
        top = z.max(axis=1, keepdims=True)
        lse = (top + np.log(np.exp(z - top).sum(axis=1, keepdims=True)))[:, 0]
        p = np.exp(z - lse[:, None])
        for t in toks:
            for e in ids[t]:
                if 0 <= e < Ne:
                    counts[gi, e] += 1
        f = counts[gi] * Ne / (k * len(toks))
        P = p.mean(axis=0)
        fd = np.zeros(n_vdev)
        h = coef * f
        for d in range(n_vdev):
            on = np.flatnonzero(np.asarray(expert_to_vdev) == d)
            if len(on):
                fd[d] = f[on].mean()
                device += fd[d] * P[on].sum() / A
                h[on] += coef_dev * fd[d]
        expert += (f * P).sum() / A
        z2 += (lse ** 2).sum() / N
        h = h / (A * len(toks))
        dlogits[toks] = p * (h - (p * h).sum(axis=1, keepdims=True)) \
            + 2 * coef_z / N * lse[:, None] * p
    total = coef * expert + coef_dev * device + coef_z * z2
    return np.array([total, expert, device, z2]), counts, dlogits
