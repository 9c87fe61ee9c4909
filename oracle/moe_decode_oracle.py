"""Oracle of nvfp4_moe_w4a16_decode: routing from the router's logits in
float64, then the expert layer of oracle.nvfp4_moe_oracle without any
intermediate rounding, and the bound of the fused computation."""

from __future__ import annotations

import numpy as np

from oracle import nvfp4_moe_oracle as MO

U = 2.0 ** -24


def route(logits, topk, scoring="softmax", renormalize=True, bias=None, weight_scale=1.0):
    """(ids [T, topk], weights [T, topk], chosen scores' distance to the next) in float64."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    for t in range(T):
        live = logits[t] > -np.inf                       # NaN and -inf are never chosen
        l = np.where(live, logits[t], -np.inf)
        if not live.any():
            continue
        if scoring == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            s = np.exp(l - l.max())
            s /= s.sum()
        key = l if bias is None else np.where(live, s + bias, -np.inf)
        order = np.argsort(-key, kind="stable")
        order = order[key[order] > -np.inf][:topk]
        ids[t, :len(order)] = order
        w[t, :len(order)] = s[order]
        if renormalize and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * weight_scale


def layer(x_bits, ids, w, w13, w2):
    """(out [T, H], bound [T, H]) for given routing; ids of -1 add nothing.

    Bound: h = float32 sums of K exact products (MFMA may truncate: 2 u each);
    through silu'(g) u and silu(g); a's float32 evaluation (2^-20) and its rounding
    to a pair of bf16 values (2^-17; the pairs of f16 that other sizes take keep
    20 bits); the second product's float32 sum; the weights (48 u: a
    softmax and a division) and the weighted sum; half a bf16 step, 2^-8."""
    live = ids >= 0
    ref = MO.moe_ref(x_bits, np.where(live, ids, 0), np.where(live, w, 0.0).astype(np.float32), w13, w2)
    T, k = ids.shape
    h, a, o = ref["h"], ref["a"], ref["o"]
    i = h.shape[1] // 2
    K1 = x_bits.shape[1]
    round_a = 2.0 ** -17
    wl = np.where(live, w, 0.0)
    out = np.einsum("tj,tjh->th", wl, o.reshape(T, k, -1))
    dh = (K1 + 4) * 2 * U * ref["h_abs"]
    dg, du = dh[:, :i], dh[:, i:]
    g, u = h[:, :i], h[:, i:]
    sg = 1.0 / (1.0 + np.exp(-np.clip(g, -700, 700)))
    slope = np.abs(sg * (1.0 + g * (1.0 - sg))) + 0.1 * dg
    da = slope * np.abs(u) * dg + np.abs(MO.silu(g)) * du + dg * du + (round_a + 2.0 ** -20) * np.abs(a)
    do, mag = np.zeros_like(o), np.zeros_like(o)
    for e, rows in enumerate(ref["groups"]):
        if rows.size:
            wa = np.abs(ref["w2deq"][e])
            mag[rows] = (np.abs(a[rows]) + da[rows]) @ wa.T
            do[rows] = da[rows] @ wa.T + (i + 8) * 2 * U * mag[rows]
    bound = np.einsum("tj,tjh->th", np.abs(wl), (do + (48 + k) * U * mag).reshape(T, k, -1))
    return out, bound + 2.0 ** -8 * np.abs(out) * (1 + 2.0 ** -7)
