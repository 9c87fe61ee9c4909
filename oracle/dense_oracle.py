"""Oracle of the int8 product, the cross entropy from hidden states and the gated
feed-forward block: the definitions in float64, and bounds for what a float32
accumulating implementation with the documented bf16 roundings may be off by.

Bounds.  U = 2^-24 is half a step of float32, HALF = 2^-8 half a step of bf16.  A
product of K terms on the matrix units rounds once per four of them, perhaps
towards zero (2 U), and once for each partial sum where K is split:
    |error| <= acc(K) * sum |terms|,   acc(K) = (K / 4 + 16 + joins) * 2 U
exp and the logistic function are taken as exp2 and a reciprocal, good to 2^-21
relative plus the rounding of their argument.  A logistic value below 2^-126 (from g = -87.3
on) is a subnormal float32 and may be zero: an absolute error of 2^-126, times what it
multiplies.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

U = 2.0 ** -24
HALF = 2.0 ** -8
TINY = 2.0 ** -126          # subnormal float32 may count as zero


JOINS = 64                  # the most partial sums a product is split into


def acc(k: int, joins: int = 0) -> float:
    return (k / 4.0 + 16.0 + joins) * 2.0 * U


# ---------------------------------------------------------------------------
# int8
# ---------------------------------------------------------------------------

def int8_scale(row: np.ndarray) -> np.float32:
    amax = np.float32(np.abs(row).max()) if row.size else np.float32(0)
    if not np.isfinite(amax):
        return np.float32(np.nan)
    return max(np.float32(amax / np.float32(127.0)), np.float32(1e-12))


def int8_quantize_rows(a: np.ndarray):
    """float64 values of a bf16 matrix -> (codes int8, scales float32): the nearest code to the exact
    ratio 127 a / amax, ties to even (where the scale is the smallest one, to a / scale in float32).  A row with
    a NaN or an infinity: codes 0, scale NaN."""
    codes = np.empty(a.shape, np.int8)
    scales = np.empty(a.shape[0], np.float32)
    for i, row in enumerate(a):
        s = scales[i] = int8_scale(row)
        amax = float(np.abs(row).max()) if row.size else 0.0
        if np.isnan(s):
            codes[i] = 0
        elif np.float32(np.float32(amax) / np.float32(127.0)) > np.float32(1e-12):
            top = Fraction(amax)
            uniq = {v: round(Fraction(127) * Fraction(v) / top) for v in set(row.tolist())}  # Python rounds half to even
            codes[i] = [uniq[v] for v in row.tolist()]
        else:
            codes[i] = np.clip(np.rint(row.astype(np.float32) / s), -127, 127)
    return codes, scales


def int8_gemm(xq, sx, wq, sw, bias=None):
    """(y, bound): exact sums; the scales' product, its product with the sum, the bias and the sum's own
    conversion to float32 round four times, then the output."""
    s = xq.astype(np.int64) @ wq.astype(np.int64).T
    y = s.astype(np.float64) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    err = 4 * U * np.abs(y)
    if bias is not None:
        y = y + bias
        err = err + 2 * U * np.abs(y)
    return y, (err + HALF * (np.abs(y) + err)) * 1.001 + TINY


# ---------------------------------------------------------------------------
# Cross entropy from hidden states
# ---------------------------------------------------------------------------

def _logits(x, w, bias):
    z = x @ w.T
    e = acc(x.shape[1]) * (np.abs(x) @ np.abs(w).T)
    if bias is not None:
        z = z + bias
        e = e + 2 * U * np.abs(np.where(np.isfinite(z), z, 0.0))
    return z, e


def _row_error(z, e, top):
    """The largest error among the logits that matter to a row's sum: one more than 100 below the
    maximum adds e^-100 at most, however far its own rounding (relative to it) moves it."""
    return np.where(z > top - 100.0, e, 0.0).max(1)


def _rows(targets, v):
    return np.nonzero((targets >= 0) & (targets < v))[0]


def linear_ce(x, w, targets, bias=None):
    """loss, lse and their bounds, [M] each; rows that do not count are 0."""
    m, v = x.shape[0], w.shape[0]
    rows = _rows(targets, v)
    loss, lse, bl, be = (np.zeros(m) for _ in range(4))
    z, e = _logits(x[rows], w, bias)
    t = targets[rows]
    top = z.max(1, keepdims=True)
    safe = np.where(np.isfinite(top), top, 0.0)
    s = np.exp(z - safe).sum(1)
    with np.errstate(divide="ignore"):
        l = safe[:, 0] + np.log(s)
    zt = z[np.arange(len(rows)), t]
    loss[rows], lse[rows] = np.where(np.isneginf(zt), np.inf, l - zt), l
    # an error of e in every logit moves lse by at most the largest; the sum of float32 terms and their
    # exponentials add relative errors that the logarithm turns into absolute ones
    ez = _row_error(z, e, top) + 2.0 ** -20 + 2 * U * np.abs(np.where(np.isfinite(l), l, 0.0)) + (v / 64.0 + 300.0) * U
    bl[rows], be[rows] = e[np.arange(len(rows)), t] + ez + 4 * U * np.abs(loss[rows]), ez
    return loss, lse, bl, be


def linear_ce_backward(x, w, targets, dloss, dlse=None, bias=None):
    """((dx, dw, db), bounds of each): dz rounded to bf16 as an operand, and what rounding took from the targets' dz added
    to each result (for dw rounded to bf16 itself)."""
    m, v = x.shape[0], w.shape[0]
    k = x.shape[1]
    rows = _rows(targets, v)
    xr, t = x[rows], targets[rows]
    z, e = _logits(xr, w, bias)
    top = z.max(1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    p = np.exp(z - top)
    p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
    d = dloss[rows][:, None]
    c = d + (0.0 if dlse is None else dlse[rows][:, None])
    dz = c * p
    one = np.zeros_like(p)
    one[np.arange(len(rows)), t] = 1.0
    dz = dz - np.where(np.isneginf(z), 0.0, d * one)
    rel = e + _row_error(z, e, top)[:, None] + 2.0 ** -20 + \
        4 * U * np.abs(np.where(np.isfinite(z), z - top, 0.0)) + (v / 64.0 + 300.0) * U
    ez = np.abs(c) * p * np.expm1(np.minimum(rel, 50.0)) + 2 * U * np.abs(d) * one
    unrounded = ez + TINY
    ez = ez + HALF * (np.abs(dz) + ez) + TINY
    az = np.abs(dz) + ez
    ez = np.where(one > 0, unrounded, ez)
    dx, bx = np.zeros((m, k)), np.zeros((m, k))
    dx[rows] = dz @ w
    bx[rows] = ez @ np.abs(w) + acc(v, JOINS + 1) * (az @ np.abs(w))
    hits = one.sum(0)[:, None]                           # more terms of a row of dw
    dw = dz.T @ xr
    bw = (ez + HALF * HALF * az * one).T @ np.abs(xr) + (acc(len(rows)) + 2.0 * U * (hits + 1.0)) * (az.T @ np.abs(xr))
    db = dz.sum(0)
    bb = ez.sum(0) + acc(len(rows)) * az.sum(0)
    return (dx, dw, db), tuple(b + HALF * (np.abs(y) + b) + TINY for y, b in ((dx, bx), (dw, bw), (db, bb)))


# ---------------------------------------------------------------------------
# Gated feed-forward block
# ---------------------------------------------------------------------------

def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def gated_ffn(x, w13, w2):
    """(y, h, a) and their bounds, h = [g, u] (float32) and a (bf16) as they are kept."""
    i = w2.shape[1]
    hu = x @ w13.T
    e = acc(x.shape[1]) * (np.abs(x) @ np.abs(w13).T)
    g, u = hu[:, :i], hu[:, i:]
    eg, eu = e[:, :i], e[:, i:]
    s = sigmoid(g)
    a = g * s * u
    # |silu'| <= 1.1, |silu''| <= 0.5; the logistic function's own error, relative
    ea = (1.1 * eg + eg * eg) * (np.abs(u) + eu) + np.abs(g * s) * eu + \
        (2.0 ** -20 + 2 * U * np.abs(g)) * np.abs(a) + TINY * np.abs(g * u)
    # up to 16 tokens a enters its product as a pair of bf16: what the second leaves is half a step of half a step
    ep = ea + (HALF * HALF if x.shape[0] <= 16 else HALF) * (np.abs(a) + ea) + TINY
    ea = ea + HALF * (np.abs(a) + ea) + TINY
    y = a @ w2.T
    ey = ep @ np.abs(w2).T + acc(i, JOINS + 1) * ((np.abs(a) + ep) @ np.abs(w2).T)
    return (y, hu, a), (ey + HALF * (np.abs(y) + ey) + TINY, e + U * np.abs(hu) + TINY, ea)


def gated_ffn_backward(x, h, a, w13, w2, dy):
    """((dx, dw13, dw2), bounds) from the h and a that the forward pass kept, dg and du rounded to bf16 as operands."""
    i = w2.shape[1]
    hd = w2.shape[0]
    g, u = h[:, :i], h[:, i:]
    da = dy @ w2
    ed = acc(hd) * (np.abs(dy) @ np.abs(w2))
    s = sigmoid(g)
    silu, slope = g * s, s * (1.0 + g * (1.0 - s))
    dh = np.concatenate((da * u * slope, da * silu), 1)
    er = 2.0 ** -20 + 2 * U * np.abs(g)
    e = np.concatenate((ed * np.abs(u * slope) + np.abs(da * u) * ((s + np.abs(silu)) * 2 * er + TINY * (1 + 2 * np.abs(g))),
                        ed * np.abs(silu) + np.abs(da * silu) * er + np.abs(da * g) * TINY), 1)
    e = e + HALF * (np.abs(dh) + e) + TINY
    ah = np.abs(dh) + e
    t = x.shape[0]
    dx, bx = dh @ w13, e @ np.abs(w13) + acc(2 * i, JOINS) * (ah @ np.abs(w13))
    dw13, b13 = dh.T @ x, e.T @ np.abs(x) + acc(t) * (ah.T @ np.abs(x))
    dw2, b2 = dy.T @ a, acc(t) * (np.abs(dy).T @ np.abs(a))
    return (dx, dw13, dw2), tuple(b + HALF * (np.abs(y) + b) + TINY
                                  for y, b in ((dx, bx), (dw13, b13), (dw2, b2)))
