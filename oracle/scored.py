"""The scored router and its gradient, in fp64, one token at a time.

Scores are the logistic function or the softmax of the logits; a logit of -inf, of
fp32's lowest value or NaN switches its expert off.  Experts are chosen by score plus
bias (by logit where there is no bias) within the groups of largest worth; equal ranks
and worths go to the lower id.  Gates are the chosen scores, renormalised on request, scaled.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

LOWEST = float(np.finfo(np.float32).min)


def scores(z, sigmoid):
    """Scores of one token's logits; zero where switched off."""
    z = np.asarray(z, dtype=np.float64)
    on = z > LOWEST
    s = np.zeros(len(z))
    if sigmoid:
        small = 1.0 / (1.0 + np.exp(np.minimum(np.abs(z[on]), 700.0)))   # of -|z|
        s[on] = np.where(z[on] > 0, 1.0 - small, np.where(z[on] < -700, 0.0, small))
    elif on.any():
        e = np.exp(z[on] - z[on].max())
        s[on] = e / e.sum()
    return s, on


def worth_of(z, s, bias, best, sigmoid):
    """Worth of a group from its experts that are on: the exact sum of its best scores and biases.

    A sigmoid above a half is 1 less its complement, so that sigmoid(x) + sigmoid(-x) is 1 for
    every x.  Without a bias scores order as the logits do, which no range of numbers ends; the
    one best score of a group is then given by its logit.
    """
    if len(z) == 0:
        return -math.inf
    rank = z if bias is None else [a + b if a + b == a + b else -math.inf for a, b in zip(s, bias)]
    if best == 1 and bias is None:
        return max(z)
    terms = []
    for i in sorted(range(len(z)), key=lambda i: (-rank[i], i))[:best]:
        if sigmoid:
            rest = 1.0 / (1.0 + math.exp(abs(z[i]))) if abs(z[i]) < 700 else 0.0
            terms += [1.0, -rest] if z[i] > 0 else [rest]
        else:
            terms.append(float(s[i]))
        if bias is not None:
            terms.append(float(bias[i]))
    if not all(map(math.isfinite, terms)):
        w = sum(terms)
        return w if w == w else -math.inf
    return sum(map(Fraction, terms))


def choose(z, bias, groups, keep, best, k, sigmoid):
    """The k experts of one token; ``groups``: group of every expert."""
    s, on = scores(z, sigmoid)
    z = np.asarray(z, dtype=np.float64)
    total = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    total = np.where(np.isnan(total), -np.inf, total)
    rank = z if bias is None else total
    G = max(groups) + 1
    worth = []
    for g in range(G):
        mine = [e for e in range(len(z)) if groups[e] == g and on[e]]
        worth.append(worth_of(z[mine], s[mine], None if bias is None else [bias[e] for e in mine], best, sigmoid))
    kept = sorted(range(G), key=lambda g: (-worth[g], g))[:keep]
    level = [2 if groups[e] not in kept else 0 if on[e] else 1 for e in range(len(z))]
    order = sorted(range(len(z)), key=lambda e: (level[e], -rank[e] if level[e] == 0 else 0.0, e))
    return order[:k]


def route(logits, k, expert_to_vdev, bias=None, sigmoid=True, n_groups=1, keep=1, best=1,
          by_vdev=False, scale=1.0, renorm=True):
    """(ids [T, k], gates [T, k], vmask [T])."""
    T, Ne = logits.shape
    groups = [int(expert_to_vdev[e]) if by_vdev and n_groups > 1 else e // (Ne // n_groups)
              for e in range(Ne)]
    ids, gates, vmask = np.zeros((T, k), np.int64), np.zeros((T, k)), np.zeros(T, np.int64)
    for t in range(T):
        s, _ = scores(logits[t], sigmoid)
        ids[t] = choose(logits[t], bias, groups, keep, best, k, sigmoid)
        g = s[ids[t]]
        if renorm:
            g = g / g.sum() if g.sum() != 0 else 0.0 * g
        gates[t] = scale * g
        for e in ids[t]:
            vmask[t] |= 1 << int(expert_to_vdev[e])
    return ids, gates, vmask


def grad(logits, ids, dgates, sigmoid=True, scale=1.0, renorm=True):
    """dlogits [T, Ne] of sum dgates * gates, the choice held fixed."""
    T, Ne = logits.shape
    out = np.zeros((T, Ne))
    for t in range(T):
        s, _ = scores(logits[t], sigmoid)
        live = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < Ne]
        S = sum(s[e] for _, e in live)
        u = {j: scale * float(dgates[t, j]) for j, _ in live}
        mean = sum(u[j] * s[e] for j, e in live) / S if S else 0.0
        ds = np.zeros(Ne)   # by expert
        for j, e in live:
            ds[e] += (u[j] if not renorm else (u[j] - mean) / S if S else 0.0)
        out[t] = ds * s * (1 - s) if sigmoid else s * (ds - (ds * s).sum())
    return out


def bias_step(bias, counts, rate):
    c = np.asarray(counts, dtype=np.int64).sum(axis=0)
    return np.asarray(bias, dtype=np.float64) + rate * np.sign(c.sum() - len(c) * c)
