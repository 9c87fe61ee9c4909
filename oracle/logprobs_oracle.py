"""Oracle of the log-probability calls, in float64 from their definitions.

Rows of logits are float64 arrays holding the exact values of the bf16, f16 or
f32 inputs.  ``allowed`` is a boolean array.  A temperature that is not
greater than 0 counts as 1.  Logits of -inf and tokens that are not allowed
have probability 0 and are never alternatives; equal logits order by index.
"""

from __future__ import annotations

import numpy as np


def allowed_bits(words: np.ndarray, v: int) -> np.ndarray:
    """uint32 [M, ceil(v / 32)] -> bool [M, v]."""
    j = np.arange(v)
    return (words[:, j // 32].astype(np.uint64) >> (j % 32).astype(np.uint64)) & np.uint64(1) == 1


def scaled(x: np.ndarray, temps, allowed):
    """(logits with -inf where not allowed, the same divided by the temperature)."""
    raw = x.astype(np.float64).copy()
    if allowed is not None:
        raw[~allowed] = -np.inf
    z = raw
    if temps is not None:
        t = np.asarray(temps, np.float64)
        z = np.full_like(raw, -np.inf)                   # -inf stays so under any temperature, +inf too
        np.divide(raw, np.where(t > 0, t, 1.0)[:, None], out=z, where=raw > -np.inf)
        z[np.isnan(raw)] = np.nan
    return raw, z


def row_stats(z: np.ndarray):
    """(maximum, log of the sum relative to it, entropy) of one row; lse is the
    sum of the first two (kept apart: at the largest magnitudes their sum
    loses the second)."""
    if np.all(z == -np.inf):
        return -np.inf, 0.0, 0.0
    if np.any(np.isnan(z)) or np.any(z == np.inf):
        return np.nan, np.nan, np.nan
    m = z.max()
    live = z[z > -np.inf] - m
    e = np.exp(live)
    return m, np.log(e.sum()), np.log(e.sum()) - np.sum(e * live) / e.sum()


def forward(x, ids=None, topk=0, temps=None, allowed=None):
    raw, z = scaled(x, temps, allowed)
    m, v = z.shape
    lse, ent = np.empty(m), np.empty(m)
    lp, rank = np.zeros(m), np.zeros(m, np.int32)
    tlp, tid = np.full((m, topk), -np.inf), np.full((m, topk), -1, np.int32)
    for i in range(m):
        top, logs, ent[i] = row_stats(z[i])
        lse[i] = top + logs
        with np.errstate(invalid="ignore"):
            logp = z[i] - top - logs if top != -np.inf else np.full(v, -np.inf)
            if ids is not None and 0 <= ids[i] < v:
                lp[i] = logp[ids[i]]
                rank[i] = 1 + np.sum(raw[i] > raw[i, ids[i]])
            live = np.flatnonzero(raw[i] > -np.inf)
        order = live[np.argsort(-raw[i][live], kind="stable")][:topk]
        tid[i, :len(order)] = order
        tlp[i, :len(order)] = logp[order]
    return lp, rank, lse, ent, tlp, tid


def forward_bounds(x, temps=None, allowed=None):
    """Error bounds per row of the float32 computation: of log S (S = the sum
    relative to the maximum), of lse and of the entropy.

    u = 2^-24 is float32's unit rounding.  The difference to the maximum, the
    quotient log2(e) / T and their product leave 3 u on each scaled
    difference, the constant a quarter more, 4 u in all; a hardware 2^y is within 2 u; a lane adds
    ceil(V / 256) terms one by one (at worst u each), may rescale its sums at
    every 16th (4 u), and the lanes join in fewer than 20 steps."""
    u = 2.0 ** -24
    _, z = scaled(x, temps, allowed)
    m, v = z.shape
    b_s, b_lse, b_h = np.empty(m), np.empty(m), np.empty(m)
    for i in range(m):
        live = z[i][z[i] > -np.inf]
        if live.size == 0 or not np.all(np.isfinite(live)):
            b_s[i] = b_lse[i] = b_h[i] = 0.0
            continue
        top = live.max()
        d = np.minimum(top - live, 104.0)                # beyond it 2^y is below float32
        e = np.exp(-d)
        mean_d = np.sum(e * d) / np.sum(e)
        rel = (v / 256.0 + v / 1024.0 + 40.0) * u + 4.0 * u * mean_d
        lse = abs(top + np.log(e.sum()))
        b_s[i] = rel
        b_lse[i] = rel + 3.0 * u * (abs(top) + lse)
        b_h[i] = 2.0 * rel * (1.0 + mean_d) + 4.0 * u * (abs(np.log(e.sum())) + mean_d)
    return b_s, b_lse, b_h


def backward(x, ids, lse, ent, dlp=None, dent=None, dlse=None, temps=None, allowed=None):
    """(gradient, the sum of its terms' magnitudes) with lse and entropy as given."""
    raw, z = scaled(x, temps, allowed)
    m, v = z.shape
    t = np.ones(m) if temps is None else np.where(np.asarray(temps, np.float64) > 0, temps, 1.0).astype(np.float64)
    g, mag = np.zeros((m, v)), np.zeros((m, v))
    for i in range(m):
        if lse[i] == -np.inf:
            continue
        given = ids is not None and 0 <= ids[i] < v and dlp is not None
        a = float(dlp[i]) if given else 0.0
        h = float(dent[i]) if dent is not None else 0.0
        s = float(dlse[i]) if dlse is not None else 0.0
        live = ~(raw[i] == -np.inf)
        logp = np.where(live, z[i] - lse[i], 0.0)
        p = np.where(live, np.exp(logp), 0.0)
        g[i] = p * (s - a)
        mag[i] = p * (abs(s) + abs(a))
        if dent is not None:
            g[i] -= h * p * (logp + ent[i])
            mag[i] += abs(h) * p * (np.abs(logp) + abs(ent[i]))
        if given and live[ids[i]]:
            g[i, ids[i]] += a
            mag[i, ids[i]] += abs(a)
        g[i] /= t[i]
        mag[i] /= t[i]
    return g, mag
