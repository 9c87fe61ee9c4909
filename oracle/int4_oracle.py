"""Oracle of the int4 group-scaled product, in float64 from its definition."""

from __future__ import annotations

import numpy as np


def unpack(words: np.ndarray, axis: int) -> np.ndarray:
    """int32 words -> the eight 4-bit values of each, low bits first, along `axis`."""
    w = words.astype(np.int64) & 0xFFFFFFFF
    q = np.stack([(w >> (4 * b)) & 15 for b in range(8)], axis=axis + 1)
    shape = list(words.shape)
    shape[axis] *= 8
    return q.reshape(shape)


def pack(q: np.ndarray, axis: int) -> np.ndarray:
    shape = list(q.shape)
    shape[axis:axis + 1] = [shape[axis] // 8, 8]
    q = np.moveaxis(q.reshape(shape).astype(np.uint64), axis + 1, -1)
    return (q << (4 * np.arange(8, dtype=np.uint64))).sum(-1).astype(np.uint32).view(np.int32)


def weight(packed, scales, zeros, n):
    """[N, K] float64 weight and the offsets [N, G]."""
    q = unpack(packed, 1).astype(np.float64)
    g = scales.shape[1]
    z = np.full((n, g), 8.0) if zeros is None else unpack(zeros, 0)[:n].astype(np.float64)
    rep = q.shape[1] // g
    return (q - np.repeat(z, rep, 1)) * np.repeat(scales.astype(np.float64), rep, 1), z


def gemm(x, packed, scales, zeros=None, bias=None):
    """(y, bound) in float64.  The bound holds the float32 summation: within a
    group partial sums of x * (16 + code) stay below 4 * 31 * ||x_group|| for
    zero-mean x, MFMA rounds (perhaps toward zero: 2 u) once per four products,
    sum x likewise; then three roundings of each group's term; the output's
    bf16 rounding is half a step, 2^-8 of the value."""
    n = packed.shape[0]
    w, _ = weight(packed, scales, zeros, n)
    y = x @ w.T
    m, k = x.shape
    g = scales.shape[1]
    size = k // g
    u = 2.0 ** -24
    xn = np.linalg.norm(x.reshape(m, g, size), axis=2)
    s = np.abs(scales.astype(np.float64))
    bound = 2.0 * (size / 4.0 + 8.0) * 2.0 * u * 4.0 * 31.0 * (xn @ s.T)
    bound += (g + 4) * u * (np.abs(x) @ np.abs(w).T)
    if bias is not None:
        y = y + bias
        bound += 2 * u * np.abs(bias)
    return y, bound + 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -7)
