"""CPU oracle of the optimizer step around the layer, in float64 (numpy).

TEST INFRASTRUCTURE, as ``moe_oracle``: the library shares no code with it.  AdamW is I. Loshchilov
and F. Hutter's "Decoupled Weight Decay Regularization"; the 8-bit states are OCP Microscaling blocks
(E4M3 elements, one power of two per 32) of m and sqrt(v), rounded at random with bits that the seed,
the step and the element's counter give (MurmurHash3's 32-bit finaliser, A. Appleby).
"""
from __future__ import annotations

import numpy as np

ODD = np.array([0x9E3779B1, 0x85EBCA77, 0xC2B2AE3D, 0x27D4EB2F, 0x165667B1, 0xD3A2646D, 0xFD7046C5, 0xB55A4F09],
               dtype=np.uint64)
LOW = np.uint64(0xFFFFFFFF)


def grad_norm(grads, max_norm):
    """(2-norm of all gradients, clip factor); the factor is NaN where the norm is not finite."""
    n = np.sqrt(sum(float(np.sum(np.square(g.astype(np.float64)))) for g in grads))
    return n, (min(1.0, max_norm / (n + 1e-6)) if np.isfinite(n) else np.nan)


def adamw(p, g, m, v, *, lr, beta1, beta2, eps, weight_decay, step, scale=1.0):
    """(p, m, v) after one step."""
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    update = (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps) + weight_decay * p
    return p - lr * update, m, v


def rounding_bits(n, counter, seed, step):
    """The 32 bits of elements counter .. counter + n - 1 (uint64 holding 32 bits each)."""
    s = np.uint64((seed ^ (step * 0x9E3779B1)) & 0xFFFFFFFF)
    i = np.arange(n, dtype=np.uint64) + np.uint64(counter)
    group = i >> np.uint64(3)
    x = (group & LOW) ^ (((group >> np.uint64(32)) * np.uint64(0x9E3779B1)) & LOW) ^ s
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x85EBCA6B)) & LOW
    x = ((x ^ (x >> np.uint64(13))) * np.uint64(0xC2B2AE35)) & LOW
    x = x ^ (x >> np.uint64(16))
    return (x * ODD[(i & np.uint64(7)).astype(np.int64)]) & LOW


def grid(y):
    """Spacing of the E4M3 grid at |y|: a 3-bit mantissa, 2^-9 below 2^-6."""
    _, e = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))
    return np.exp2(e - 4.0)


def scale_exponent(block_max):
    """Exponent of the least power of two with block_max <= 448 * 2^x, in [-126, 127]."""
    with np.errstate(divide="ignore"):
        x = np.ceil(np.log2(block_max / 448.0))
    return np.clip(np.where(block_max > 0, x, -126), -126, 127)


def to_mx8(t, bits, root):
    """(E4M3 values, exponents) of a float64 vector in blocks of 32.  ``root``: the rule for sqrt(v), which
    takes the low 23 bits and never becomes zero; m takes the high 23."""
    n = t.size
    pad = np.zeros(-(-n // 32) * 32)
    pad[:n] = t
    x = scale_exponent(np.abs(pad).reshape(-1, 32).max(axis=1))
    y = t / np.exp2(np.repeat(x, 32)[:n])
    u = ((bits & np.uint64(0x7FFFFF)) if root else (bits >> np.uint64(9))).astype(np.float64) * 2.0 ** -23
    q = np.floor(y / grid(y) + u) * grid(y)
    if root:
        q = np.where(y > 0, np.maximum(q, 2.0 ** -9), q)
    return np.clip(q, -448, 448), x


def to_bf16_random(p, bits):
    """float32 values of a bf16 rounding that goes up with the probability of the part cut off."""
    b = p.astype(np.float32).view(np.uint32).astype(np.uint64)
    return (((b + (bits & np.uint64(0xFFFF))) & LOW & np.uint64(0xFFFF0000)).astype(np.uint32)).view(np.float32)
