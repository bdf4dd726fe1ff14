"""64-bit oracle of the token embedding and of microscaled 4-bit floating point
("OCP Microscaling Formats (MX) Specification" v1.0: E2M1 elements, blocks of
32, E8M0 scales), in numpy.
"""
from __future__ import annotations

import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def embedding(tokens, weight, scale=1.0):
    """scale * weight[tokens], zero rows for tokens outside the vocabulary."""
    tokens = np.asarray(tokens)
    out = np.zeros(tokens.shape + weight.shape[1:])
    for at in np.ndindex(tokens.shape):
        if 0 <= tokens[at] < weight.shape[0]:
            out[at] = scale * weight[tokens[at]]
    return out


def embedding_grad(tokens, grad, vocab, scale=1.0, old=None):
    """(gradient, sums of magnitudes, number of terms of every row)."""
    width = grad.shape[-1]
    tokens, grad = np.asarray(tokens).reshape(-1), grad.reshape(-1, width)
    sums, sizes, n = np.zeros((vocab, width)), np.zeros((vocab, width)), np.zeros(vocab, dtype=int)
    for t, g in zip(tokens.tolist(), grad):
        if 0 <= t < vocab:
            sums[t] += g
            sizes[t] += np.abs(g)
            n[t] += 1
    sums, sizes = sums * scale, sizes * abs(scale)
    if old is not None:
        sums, sizes = sums + old, sizes + np.abs(old)
    return sums, sizes, n


def mxfp4_quantize(x, noise=None):
    """(codes, scales) of float64 x [..., cols], one code per element and one
    scale byte per block."""
    lead, cols = x.shape[:-1], x.shape[-1]
    blocks = -(-cols // 32)
    codes, scales = np.zeros(x.shape, dtype=np.uint8), np.zeros(lead + (blocks,), dtype=np.uint8)
    for at in np.ndindex(*lead, blocks):
        sel = at[:-1] + (slice(32 * at[-1], min(cols, 32 * at[-1] + 32)),)
        v = x[sel]
        if not np.isfinite(v).all():
            scales[at] = 255
            continue
        largest = float(np.max(np.abs(v)))
        exponent = math.frexp(largest)[1] - 1 - 2 if largest > 0 else -127   # floor(log2) - 2
        exponent = max(exponent, -127)
        if noise is not None and largest > 6 * math.ldexp(1.0, exponent):
            exponent += 1
        scales[at] = exponent + 127
        t = np.abs(v) / math.ldexp(1.0, exponent)
        low = np.searchsorted(GRID, t, side="right") - 1
        high = np.minimum(low + 1, 7)
        gap = np.where(low < 7, GRID[high] - GRID[low], 1.0)
        f = np.minimum((t - GRID[low]) / gap, 1.0)
        if noise is None:
            up = (f > 0.5) | ((f == 0.5) & (low % 2 == 1))
        else:
            up = 256 * f > noise[sel].astype(np.float64) + 0.5
        code = np.where(low < 7, low + up, 7).astype(np.uint8)
        codes[sel] = code | (np.signbit(v).astype(np.uint8) << 3)
    return codes, scales


def mxfp4_values(codes, scales):
    """The values that codes and scale bytes stand for."""
    value = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    s = np.repeat(scales, 32, axis=-1)[..., :codes.shape[-1]].astype(np.int64)
    return np.where(s == 255, np.nan, np.ldexp(value, s - 127))
