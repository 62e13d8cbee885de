"""CPU oracle of the operators for experts outside the layer, in float64 (numpy): rows by a schedule table, E4M3
quantisation in blocks of 128, the grouped product and its weight gradient.

TEST INFRASTRUCTURE, as ``moe_oracle``: the library shares no code with it.
"""
from __future__ import annotations

import numpy as np

TOP, LEAST = 448.0, 2.0 ** -110


def table(expert, E):
    """src_of, row_of, offsets of assignments' experts (-1: dropped), one after the other; empty rows at the end."""
    n = len(expert)
    src, row, offsets = np.full(n, -1, np.int32), np.full(n, -1, np.int32), np.zeros(E + 1, np.int32)
    r = 0
    for e in range(E):
        for a in range(n):
            if expert[a] == e:
                src[r], row[a] = a, r
                r += 1
        offsets[e + 1] = r
    return src, row, offsets


def gather(x, src_of, k, gates=None):
    out = np.zeros((len(src_of), x.shape[1]))
    for r, a in enumerate(src_of):
        if a >= 0:
            out[r] = x[a // k] * (1.0 if gates is None else gates[a // k, a % k])
    return out


def merge(o, row_of, k, gates=None):
    """(y, the sum of the terms' magnitudes)"""
    T = len(row_of) // k
    y, size = np.zeros((T, o.shape[1])), np.zeros((T, o.shape[1]))
    for a, r in enumerate(row_of):
        if r >= 0:
            term = o[r] * (1.0 if gates is None else gates[a // k, a % k])
            y[a // k] += term
            size[a // k] += np.abs(term)
    return y, size


def merge_backward(dy, o, row_of, gates):
    """(do with NaN in rows that no assignment names, dgates, the dot products' sums of magnitudes)"""
    T, k = gates.shape
    do, dg, size = np.full(o.shape, np.nan), np.zeros((T, k)), np.zeros((T, k))
    for a, r in enumerate(row_of):
        if r >= 0:
            t, j = divmod(a, k)
            do[r] = gates[t, j] * dy[t]
            dg[t, j] = dy[t] @ o[r]
            size[t, j] = np.abs(dy[t]) @ np.abs(o[r])
    return do, dg, size


def silu(h):
    with np.errstate(over="ignore"):
        return h / (1.0 + np.exp(-h))


def swiglu(x):
    """(a, the size of its rounding errors' terms)"""
    h, u = np.split(x, 2, axis=1)
    a = silu(h) * u
    return a, np.abs(a)


def swiglu_grad(x, da):
    """dh | du of a = silu(h) u, and the size of the terms"""
    h, u = np.split(x, 2, axis=1)
    with np.errstate(over="ignore"):
        sg = 1.0 / (1.0 + np.exp(-h))
    dh, du = da * u * (sg + h * sg * (1.0 - sg)), da * h * sg
    return np.concatenate([dh, du], 1), np.concatenate([np.abs(da * u * sg) * (1.0 + np.abs(h)), np.abs(du)], 1)


def e4m3(y):
    """The E4M3 value nearest to y, ties to even."""
    _, exponent = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))
    step = np.exp2(exponent - 4.0)
    return np.clip(np.round(y / step) * step, -TOP, TOP)


def e4m3_step(y):
    """The distance of the E4M3 values around y."""
    _, exponent = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))
    return np.exp2(exponent - 4.0)


def largest(x, axis):
    """The blocks' largest finite magnitudes, at least LEAST."""
    m = np.where(np.isfinite(x), np.abs(x), 0.0)
    return np.maximum(m.max(axis=axis, initial=0.0), LEAST)


def rows(x):
    """(448 x / amax with amax of each 128 along the row, scales [blocks][R])"""
    y, scales = np.zeros(x.shape), []
    for c in range(0, x.shape[1], 128):
        m = largest(x[:, c:c + 128], 1)
        y[:, c:c + 128] = x[:, c:c + 128] * TOP / m[:, None]
        scales.append(m / TOP)
    return y, np.array(scales)


def columns(x, offsets):
    """(the transposed layout, 448 x / amax with amax of each 128 rows of a group; scales [P/128][C], NaN behind the last
    block)"""
    E, (R, C) = len(offsets) - 1, x.shape
    blocks = R // 128 + E
    y, scales = np.full((C, 128 * blocks), np.nan), np.full((blocks, C), np.nan)
    b = 0
    for e in range(E):
        for r in range(offsets[e], offsets[e + 1], 128):
            part = x[r:min(r + 128, offsets[e + 1])]
            m = largest(part, 0)
            y[:, 128 * b:128 * (b + 1)] = 0.0
            y[:, 128 * b:128 * b + len(part)] = (part * TOP / m).T
            scales[b] = m / TOP
            b += 1
    return y, scales


def weights(w):
    """(448 w / amax, scales [E][N/128][K/128])"""
    y, E = np.zeros(w.shape), w.shape[0]
    n, k = -(-w.shape[1] // 128), -(-w.shape[2] // 128)
    scales = np.zeros((E, n, k))
    for e in range(E):
        for i in range(n):
            for j in range(k):
                part = w[e, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                m = largest(part, None)
                y[e, 128 * i:128 * i + 128, 128 * j:128 * j + 128] = part * TOP / m
                scales[e, i, j] = m / TOP
    return y, scales


def product(x, x_scale, w, w_scale, offsets):
    """(out with NaN in rows of no group, the sum of the terms' magnitudes)"""
    R, K, N = x.shape[0], x.shape[1], w.shape[1]
    xs = np.repeat(x_scale, 128, 0)[:K].T * x
    out, size = np.full((R, N), np.nan), np.zeros((R, N))
    for e in range(w.shape[0]):
        ws = np.repeat(np.repeat(w_scale[e], 128, 0), 128, 1)[:N, :K] * w[e]
        cut = slice(offsets[e], offsets[e + 1])
        out[cut] = xs[cut] @ ws.T
        size[cut] = np.abs(xs[cut]) @ np.abs(ws).T
    return out, size


def weight_grad(dy, dy_scale, x, x_scale, offsets):
    E = len(offsets) - 1
    out, size = np.zeros((E, dy.shape[0], x.shape[0])), np.zeros((E, dy.shape[0], x.shape[0]))
    b = 0
    for e in range(E):
        for _ in range(offsets[e], offsets[e + 1], 128):
            p = dy[:, 128 * b:128 * b + 128] * dy_scale[b][:, None]
            q = x[:, 128 * b:128 * b + 128] * x_scale[b][:, None]
            out[e] += p @ q.T
            size[e] += np.abs(p) @ np.abs(q).T
            b += 1
    return out, size
