"""CPU oracle of group-limited expert selection, its balance terms and its backward, in float64 (numpy).

TEST INFRASTRUCTURE, as ``moe_oracle``: the library shares no code with it.  The rule is DeepSeek-V3's
node-limited routing (groups ranked by the sum of their two best biased scores) with its softmax
predecessor (groups ranked by their best), a bias that moves the selection only, and the balance loss
coef * E / (k T^2) * sum_e counts[e] * prob_sum[e].  One token at a time, by Python's own sort.
"""
from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1


def scores(x, router):
    """[T][E] scores of float64 logits; a row of -inf has softmax scores 0."""
    with np.errstate(invalid="ignore", over="ignore"):
        if router == SIGMOID:
            return 1.0 / (1.0 + np.exp(-x))
        m = x.max(axis=1, keepdims=True)
        e = np.exp(x - np.where(np.isfinite(m), m, 0.0))
        total = e.sum(axis=1, keepdims=True)
        return e / np.where(total == 0, 1.0, total)


def select(x, bias, router, k, n_group, topk_group, group_score):
    """(topk_idx [T][k], margin [T]): the margin is the least distance between two values whose order
    decided the selection or its order (group values at the cut, rank values down to the first one left)."""
    T, E = x.shape
    s = scores(x, router)
    size = E // n_group
    idx, margins = np.zeros((T, k), np.int32), np.zeros(T)
    for t in range(T):
        by_logit = router == SOFTMAX and bias is None
        alive = x[t] > -np.inf                     # neither -inf nor NaN
        rank = x[t] if by_logit else s[t] + (0.0 if bias is None else bias)
        rank = np.where(alive, rank, -np.inf)
        pair = np.where(alive, s[t], -np.inf) if by_logit and group_score == GROUP_TOP2 else rank
        margin = np.inf
        experts = range(E)
        if n_group > 1:
            value = []
            for g in range(n_group):
                best = sorted((pair[e] for e in range(g * size, (g + 1) * size) if alive[e]), reverse=True)
                value.append(-np.inf if not best else best[0] if group_score == GROUP_MAX else sum(best[:2]))
            order = sorted(range(n_group), key=lambda g: (-value[g], g))
            if topk_group < n_group:
                a, b = value[order[topk_group - 1]], value[order[topk_group]]
                margin = min(margin, a - b if a > -np.inf else np.inf)
            experts = [e for g in sorted(order[:topk_group]) for e in range(g * size, (g + 1) * size)]
        order = sorted(experts, key=lambda e: (-rank[e], e))
        cut = [rank[e] for e in order[:k + 1] if rank[e] > -np.inf]
        if len(cut) > 1:
            margin = min(margin, min(a - b for a, b in zip(cut, cut[1:])))
        idx[t], margins[t] = order[:k], margin
    return idx, margins


def gates(s, idx, renorm, scale):
    g = np.take_along_axis(s, idx.astype(np.int64), axis=1)
    if renorm:
        total = g.sum(axis=1, keepdims=True)
        g = np.where(total == 0, 0.0, g / np.where(total == 0, 1.0, total))
    return g * scale


def probabilities(s):
    total = s.sum(axis=1, keepdims=True)
    return np.where(total == 0, 0.0, s / np.where(total == 0, 1.0, total))


def balance(s, idx, coef, bias, rate):
    """counts, prob_sum, loss, dprob, bias_next (None without a bias)."""
    T, E = s.shape
    k = idx.shape[1]
    counts = np.zeros(E, np.int64)
    for e in idx.ravel():
        counts[e] += 1
    prob_sum = probabilities(s).sum(axis=0)
    dprob = coef * E / (k * T * T) * counts if T else np.zeros(E)
    moved = None if bias is None else bias + rate * np.sign(T * k - E * counts)
    return counts, prob_sum, float(dprob @ prob_sum), dprob, moved


def backward(x, idx, dgates, dprob, router, renorm, scale):
    """dlogits: the chain rule with the Jacobians written out, one token at a time."""
    T, E = x.shape
    s = scores(x, router)
    out = np.zeros((T, E))
    for t in range(T):
        ds = np.zeros(E)
        if dgates is not None:
            sel = s[t, idx[t]]
            S = sel.sum()
            for j, e in enumerate(idx[t]):
                for i in range(len(sel)):           # d gate_i / d s_j
                    if not renorm:
                        d = scale * (i == j)
                    else:
                        d = 0.0 if S == 0 else scale * ((i == j) / S - sel[i] / S ** 2)
                    ds[e] += dgates[t, i] * d
        if dprob is not None:
            total = s[t].sum()
            if total > 0:
                ds += dprob / total - (dprob * s[t]).sum() / total ** 2
        if router == SIGMOID:
            out[t] = ds * s[t] * (1 - s[t])
        else:
            out[t] = s[t] * (ds - (s[t] * ds).sum())
    return out
