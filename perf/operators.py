"""What is measured of the decode-tail operators: the expert layer of a few
tokens, the int4 group-scaled product that gives logits, the log probabilities
of given tokens and their gradient.

``run`` computes each operator in its plain form (elementary torch operations
in float32) or, where ``own`` is true, through the library's entry points.
``exact`` computes the same outputs from the definitions in float64.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f16": 2, "f32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _lp(name, m, v, dtype, topk, temps=False, mask=False, pad=0):
    return {"name": name, "op": "logprobs", "M": m, "V": v, "dtype": dtype, "topk": topk, "temps": temps,
            "mask": mask, "pad": pad}


def _lpb(name, m, v, dtype, entropy=True, temps=False, mask=False, pad=0):
    return {"name": name, "op": "logprobs_backward", "M": m, "V": v, "dtype": dtype, "entropy": entropy,
            "temps": temps, "mask": mask, "pad": pad}


def _moe(name, t, e, topk, h, i, scoring="softmax", renorm=True):
    return {"name": name, "op": "moe_decode", "T": t, "E": e, "topk": topk, "H": h, "I": i, "scoring": scoring,
            "renorm": renorm}


def _i4(name, m, n, k, group, zeros, bias=False):
    return {"name": name, "op": "int4_gemm", "M": m, "N": n, "K": k, "group": group, "zeros": zeros, "bias": bias}


def listed():
    return [
        # one new token of one sequence, reported with its five best alternatives: latency
        _lp("logprobs_1x128256", 1, 128256, "bf16", 5),
        # a decode batch under a grammar: sampling temperatures, a mask of the allowed tokens
        _lp("logprobs_64x151936_masked", 64, 151936, "bf16", 20, temps=True, mask=True),
        # scoring a prompt: every position's own token and the best alternative
        _lp("logprobs_2048x128256", 2048, 128256, "bf16", 1),
        # float32 logits of an odd vocabulary in a wider buffer, most alternatives
        _lp("logprobs_333x32003_f32", 333, 32003, "f32", 64, temps=True, pad=5),
        # a policy-gradient step with an entropy bonus
        _lpb("logprobs_backward_1024x128256", 1024, 128256, "bf16", temps=True),
        # a short f16 answer of an odd vocabulary (rows of every alignment), no entropy term
        _lpb("logprobs_backward_17x32003_f16", 17, 32003, "f16", entropy=False),
        # one token through the repository's expert layer
        _moe("moe_1_8x4096", 1, 8, 2, 4096, 14336),
        # a decode batch of 16 through the same layer: every expert is read
        _moe("moe_16_8x4096", 16, 8, 2, 4096, 14336),
        # many small experts, sigmoid scores, a few tokens
        _moe("moe_4_64x2048", 4, 64, 6, 2048, 1024, "sigmoid"),
        # one token's logits from an int4 lm_head with groups of 128
        _i4("int4_1x128256x4096", 1, 128256, 4096, 128, False),
        # a batch of 16 over the widest head, zero points
        _i4("int4_16x151936x5120", 16, 151936, 5120, 128, True),
        # a ragged batch, odd vocabulary, the smallest groups, zero points and bias
        _i4("int4_33x32003x2080", 33, 32003, 2080, 32, True, True),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm, odd ones among them."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_backward", "moe_decode", "int4_gemm"])
    if op in ("logprobs", "logprobs_backward"):
        v = _log_int(rng, 1000, 152000)
        dtype = rng.choice(["bf16", "f16", "f32"])
        # at most the largest listed case's bytes
        cap = 2048 * 128256 * 2 if op == "logprobs" else 1024 * 128256 * 2
        m = _log_int(rng, 1, max(1, min(2048, cap // (v * ESIZE[dtype]))))
        temps, mask, pad = rng.random() < 0.5, rng.random() < 0.3, rng.choice([0, 0, 3, 8])
        if op == "logprobs":
            case = _lp("", m, v, dtype, rng.choice([0, 1, 5, 20, 33, 64]), temps, mask, pad)
        else:
            case = _lpb("", m, v, dtype, rng.random() < 0.6, temps, mask, pad)
    elif op == "moe_decode":
        e = rng.choice([4, 8, 16, 60, 64, 128])
        topk = rng.randint(1, min(8, e // 2))
        h = 16 * _log_int(rng, 32, 448)
        cap = 8 * 3 * 4096 * 14336
        i = 16 * _log_int(rng, 16, max(16, min(896, cap // (16 * 3 * e * h))))
        case = _moe("", rng.randint(1, 16), e, topk, h, i, rng.choice(["softmax", "softmax", "sigmoid"]),
                    rng.random() < 0.7)
    else:
        group = rng.choice([32, 64, 128])
        k = 128 * _log_int(rng, 4, 64) + (group if group < 128 and rng.random() < 0.3 else 0)
        n = _log_int(rng, 1000, max(1000, min(152000, 151936 * 5120 // k)))
        case = _i4("", rng.choice([1, 2, 3, 5, 8, 13, 16, 24, 33, 64]), n, k, group, rng.random() < 0.5,
                   rng.random() < 0.3)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _logits(case, g):
    """Logits as a language model gives them: a broad bulk and, in each row, a
    few tokens far above it."""
    m, v, pad = case["M"], case["V"], case["pad"]
    dtype = DTYPES[case["dtype"]]
    buf = torch.empty((m, v + pad), dtype=dtype, device=DEV)
    rows = max(1, (1 << 26) // (v + pad))
    for r in range(0, m, rows):
        n = min(rows, m - r)
        buf[r:r + n] = (2.5 * torch.randn((n, v + pad), generator=g, device=DEV)).to(dtype)
    x = buf[:, :v]
    few = torch.randint(0, v, (m, 1), generator=g, device=DEV)
    few = (few + v // 12 * torch.arange(12, device=DEV)) % v             # distinct in a row
    high = 7.0 + 3.0 * torch.randn((m, 12), generator=g, device=DEV)
    x.scatter_(1, few, high.to(dtype))
    # the given token: a likely one in most rows, any other one in the rest
    tok = torch.where(torch.rand((m,), generator=g, device=DEV) < 0.7, few[:, 0],
                      torch.randint(0, v, (m,), generator=g, device=DEV))
    temps = None
    if case["temps"]:
        temps = 0.6 + 0.7 * torch.rand((m,), generator=g, device=DEV)
    allowed = None
    if case["mask"]:
        words = (v + 31) // 32
        draw1 = torch.randint(-2 ** 31, 2 ** 31, (m, words), generator=g, device=DEV, dtype=torch.int64)
        draw2 = torch.randint(-2 ** 31, 2 ** 31, (m, words), generator=g, device=DEV, dtype=torch.int64)
        allowed = (draw1 & draw2).to(torch.int32)            # a quarter of the tokens
        for t in [tok] + [few[:, j] for j in range(12)]:     # the likely ones among them
            w = (t // 32).unsqueeze(1)
            bit = torch.bitwise_left_shift(torch.ones_like(t), t % 32).unsqueeze(1)
            bit = torch.where(bit >= 2 ** 31, bit - 2 ** 32, bit).to(torch.int32)
            allowed.scatter_(1, w, allowed.gather(1, w) | bit)
    return x, tok.to(torch.int32), temps, allowed


def _nvfp4_experts(e, n, k, g):
    """Expert weights N(0, 0.02) in the NVFP4 layout: packed codes, E4M3 block
    scales, one global scale per expert."""
    packed = torch.empty((e, n, k // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((e, n, k // 16), dtype=torch.float8_e4m3fn, device=DEV)
    gs = torch.empty((e,), dtype=torch.float32, device=DEV)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for i in range(e):
        w = 0.02 * torch.randn((n, k // 16, 16), generator=g, device=DEV)
        gs[i] = w.abs().amax() / 2688.0
        s = (w.abs().amax(2) / 6.0 / gs[i]).to(torch.float8_e4m3fn)
        scales[i] = s
        q = w / (s.float() * gs[i]).clamp_min(1e-20).unsqueeze(2)
        code = torch.bucketize(q.abs(), mids).to(torch.uint8)
        code += 8 * ((q < 0) & (code > 0)).to(torch.uint8)
        code = code.view(n, k // 2, 2)
        packed[i] = code[:, :, 0] | (code[:, :, 1] << 4)
    return packed, scales, gs


def _int4_weight(n, k, group, zeros, g):
    """Weights N(0, 0.02) in the int4 group layout: eight codes per int32 along
    K, bfloat16 scales, zero points packed eight rows to an int32."""
    packed = torch.empty((n, k // 8), dtype=torch.int32, device=DEV)
    scales = torch.empty((n, k // group), dtype=torch.bfloat16, device=DEV)
    ng = k // group
    zp = torch.zeros(((n + 7) // 8 * 8, ng), dtype=torch.int64, device=DEV)
    shift = 4 * torch.arange(8, device=DEV)
    rows = max(8, (1 << 26) // k // 8 * 8)
    for r in range(0, n, rows):
        c = min(rows, n - r)
        w = 0.02 * torch.randn((c, ng, group), generator=g, device=DEV)
        if zeros:
            lo, hi = w.amin(2), w.amax(2)
            s = ((hi - lo) / 15.0).to(torch.bfloat16)
            z = torch.round(-lo / s.float()).clamp_(0, 15)
            zp[r:r + c] = z.to(torch.int64)
        else:
            s = (w.abs().amax(2) / 7.5).to(torch.bfloat16)
            z = torch.full_like(s, 8.0, dtype=torch.float32)
        scales[r:r + c] = s
        code = (torch.round(w / s.float().unsqueeze(2)) + z.unsqueeze(2)).clamp_(0, 15).to(torch.int64)
        word = (code.view(c, k // 8, 8) << shift).sum(2)
        packed[r:r + c] = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)
    if not zeros:
        return packed, scales, None
    word = (zp.view(-1, 8, ng) << shift.view(1, 8, 1)).sum(1)
    return packed, scales, torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("logprobs", "logprobs_backward"):
        st["x"], st["tok"], st["temps"], st["allowed"] = _logits(case, g)
        if op == "logprobs_backward":
            m = case["M"]
            # what the forward pass left behind, and the gradients that the loss sends back
            # (in float16 with the loss scale that keeps small gradients out of its subnormals)
            st["lse"], st["entropy"] = (t.float() for t in _stats64(st))
            scale = (4096.0 if case["dtype"] == "f16" else 1.0) / m
            st["dlp"] = scale * torch.randn((m,), generator=g, device=DEV)
            st["dent"] = 0.01 * scale * torch.randn((m,), generator=g, device=DEV) if case["entropy"] else None
    elif op == "moe_decode":
        t, e, h, i = case["T"], case["E"], case["H"], case["I"]
        st["x"] = torch.randn((t, h), generator=g, device=DEV).to(torch.bfloat16)
        st["router"] = 1.5 * torch.randn((t, e), generator=g, device=DEV)
        st["w13"] = _nvfp4_experts(e, 2 * i, h, g)
        st["w2"] = _nvfp4_experts(e, h, i, g)
    else:
        n, k = case["N"], case["K"]
        st["x"] = torch.randn((case["M"], k), generator=g, device=DEV).to(torch.bfloat16)
        st["packed"], st["scales"], st["zp"] = _int4_weight(n, k, case["group"], case["zeros"], g)
        st["bias"] = None
        if case["bias"]:
            st["bias"] = (0.5 * torch.randn((n,), generator=g, device=DEV)).to(torch.bfloat16)
    if own:
        # the output buffers and workspace that a serving loop keeps
        from nvfp4_w4a16_lm_amd import binding as B
        if op == "logprobs":
            st["out"] = B.logprobs_buffers(case["M"], case["V"], case["topk"], DEV)
        elif op == "moe_decode":
            st["ws"] = B.moe_decode_workspace(case["T"], case["topk"], case["E"], case["H"], case["I"], DEV)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _run_own(st):
    from nvfp4_w4a16_lm_amd import binding as B
    case = st["case"]
    op = case["op"]
    if op == "logprobs":
        r = B.nvfp4_logprobs(st["x"], st["tok"], topk=case["topk"], temperatures=st["temps"],
                             allowed=st["allowed"], out=st["out"])
        return tuple(r[:6])
    if op == "logprobs_backward":
        return B.nvfp4_logprobs_backward(st["x"], st["tok"], st["lse"], st["entropy"], st["dlp"],
                                         dentropy=st["dent"], temperatures=st["temps"], allowed=st["allowed"])
    if op == "moe_decode":
        return B.nvfp4_moe_w4a16_decode(st["x"], st["router"], case["topk"], st["w13"], st["w2"],
                                        scoring=case["scoring"], renormalize=case["renorm"], workspace=st["ws"])
    return B.nvfp4_int4_gemm(st["x"], st["packed"], st["scales"], zero_points=st["zp"], bias=st["bias"])


def _mask_bits(allowed, v):
    bits = (allowed.unsqueeze(2) >> torch.arange(32, device=allowed.device, dtype=torch.int32)) & 1
    return bits.flatten(1)[:, :v] == 1


def _plain_logprobs(st):
    case = st["case"]
    x = st["x"].float()
    m, v = x.shape
    if st["allowed"] is not None:
        x = torch.where(_mask_bits(st["allowed"], v), x, -math.inf)
    z = x if st["temps"] is None else x / st["temps"].unsqueeze(1)
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    s = e.sum(1, keepdim=True)
    lse = top + torch.log(s)
    tok = st["tok"].long().unsqueeze(1)
    lp = z.gather(1, tok) - lse
    ent = torch.log(s) - torch.where(e > 0, e * (z - top), 0.0).sum(1, keepdim=True) / s
    rank = (x > x.gather(1, tok)).sum(1).to(torch.int32) + 1
    k = case["topk"]
    if k > 0:
        # value, then the lower index, in one whole number
        u = (x + 0.0).view(torch.int32)
        u = torch.where(u < 0, u ^ 0x7FFFFFFF, u)
        key = u.long() * (1 << 32) - torch.arange(v, device=x.device)
        ids = torch.topk(key, k, dim=1).values.neg_().bitwise_and_((1 << 32) - 1)
        tlp = z.gather(1, ids) - lse
        ids = ids.to(torch.int32)
    else:
        ids, tlp = tok[:, :0].to(torch.int32), z[:, :0]
    return lp.squeeze(1), rank, lse.squeeze(1), ent.squeeze(1), tlp, ids


def _plain_backward(st):
    x = st["x"].float()
    m, v = x.shape
    if st["allowed"] is not None:
        x = torch.where(_mask_bits(st["allowed"], v), x, -math.inf)
    z = x if st["temps"] is None else x / st["temps"].unsqueeze(1)
    lp = z - st["lse"].unsqueeze(1)
    p = torch.exp(lp)
    dz = -st["dlp"].unsqueeze(1) * p
    if st["dent"] is not None:
        dz -= st["dent"].unsqueeze(1) * torch.where(p > 0, p * (lp + st["entropy"].unsqueeze(1)), 0.0)
    dz.scatter_add_(1, st["tok"].long().unsqueeze(1), st["dlp"].unsqueeze(1))
    if st["temps"] is not None:
        dz /= st["temps"].unsqueeze(1)
    return dz.to(st["x"].dtype)


def _dequant(packed, scales, gs, dtype):
    lut = torch.tensor(E2M1, dtype=dtype, device=packed.device)
    code = torch.stack((packed & 15, packed >> 4), dim=-1).int()
    w = lut[code].view(packed.shape[0], -1, 16)
    return (w * scales.to(dtype).unsqueeze(2)).view(packed.shape[0], -1) * gs.to(dtype)


def _route(st, dtype):
    case = st["case"]
    logits = st["router"].to(dtype)
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :case["topk"]]
    if case["scoring"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-logits))
    else:
        s = torch.exp(logits - logits.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    w = s.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids, w


def _plain_moe(st):
    case = st["case"]
    e, k, i = case["E"], case["topk"], case["I"]
    x = st["x"].float()
    ids, w = _route(st, torch.float32)
    out = torch.zeros_like(x)

    def expert(xe, p13, s13, g13, p2, s2, g2):
        h = xe @ _dequant(p13, s13, g13, torch.float32).t()
        gate, up = h[:, :i], h[:, i:]
        return (gate / (1.0 + torch.exp(-gate)) * up) @ _dequant(p2, s2, g2, torch.float32).t()

    def pick(w3, j):
        return w3[0].index_select(0, j)[0], w3[1].view(torch.uint8).index_select(0, j)[0].view(w3[1].dtype), \
            w3[2].index_select(0, j)

    if case["T"] * k <= e:                               # fewer pairs than experts: one product for each pair
        for t in range(case["T"]):
            for j in range(k):
                idx = ids[t, j].reshape(1)
                out[t:t + 1] += w[t, j] * expert(x[t:t + 1], *pick(st["w13"], idx), *pick(st["w2"], idx))
    else:
        gate = torch.zeros((case["T"], e), device=x.device).scatter_(1, ids, w)
        for j in range(e):
            out += gate[:, j:j + 1] * expert(x, *(t[j] for t in st["w13"]), *(t[j] for t in st["w2"]))
    return out.to(torch.bfloat16), ids.to(torch.int32), w


def _int4_dequant(packed, scales, zp, r0, group, dtype):
    """Rows r0, ... of the weight: (code - zero) * scale."""
    n = packed.shape[0]
    shift = 4 * torch.arange(8, device=packed.device, dtype=torch.int32)
    code = ((packed.unsqueeze(2) >> shift) & 15).view(n, -1, group)
    if zp is None:
        z = 8
    else:
        rows = r0 + torch.arange(n, device=packed.device)
        z = (zp[rows // 8] >> (4 * (rows % 8)).to(torch.int32).unsqueeze(1)) & 15
        z = z.unsqueeze(2)
    return ((code - z).to(dtype) * scales.to(dtype).unsqueeze(2)).view(n, -1)


def _plain_int4(st, dtype=torch.float32, rows=None):
    case = st["case"]
    n, k = case["N"], case["K"]
    x = st["x"].to(dtype)
    y = torch.empty((case["M"], n), dtype=dtype, device=x.device)
    step = n if rows is None else rows
    for r in range(0, n, step):
        w = _int4_dequant(st["packed"][r:r + step], st["scales"][r:r + step], st["zp"], r, case["group"], dtype)
        y[:, r:r + step] = x @ w.t()
    if st["bias"] is not None:
        y += st["bias"].to(dtype)
    return y


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "logprobs":
        return _plain_logprobs(state)
    if op == "logprobs_backward":
        return _plain_backward(state)
    if op == "moe_decode":
        return _plain_moe(state)
    return _plain_int4(state).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# Work, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("logprobs", "logprobs_backward"):
        m, v = case["M"], case["V"]
        b = m * v * ESIZE[case["dtype"]] + (m * ((v + 31) // 32) * 4 if case["mask"] else 0)
        if op == "logprobs":
            return {"bytes": b + m * (20 + 8 * case["topk"]), "flops": 7 * m * v}
        return {"bytes": b + m * v * ESIZE[case["dtype"]] + 24 * m, "flops": 8 * m * v}
    if op == "moe_decode":
        t, e, k, h, i = case["T"], case["E"], case["topk"], case["H"], case["I"]
        active = e * (1.0 - (1.0 - k / e) ** t)          # experts that some token chose, on average
        return {"bytes": int(active * 3 * h * i * 0.5625) + 4 * t * h + 4 * t * e + 8 * t * k,
                "flops": 6 * t * k * h * i}
    m, n, k = case["M"], case["N"], case["K"]
    groups = n * (k // case["group"])
    b = n * k // 2 + 2 * groups + (groups // 2 if case["zeros"] else 0) + 2 * m * k + 2 * m * n
    return {"bytes": b + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}


def _rows64(st, r, n):
    """Scaled and masked logits of rows r, ..., r + n - 1 in float64."""
    x = st["x"][r:r + n].double()
    if st["allowed"] is not None:
        bit = torch.arange(x.shape[1], device=x.device)
        word = st["allowed"][r:r + n].long()[:, bit // 32]
        x.masked_fill_((word >> (bit % 32)) & 1 == 0, -math.inf)
    raw = x
    if st["temps"] is not None:
        x = x / st["temps"][r:r + n].double().unsqueeze(1)
    return raw, x


def _chunks(st):
    m, v = st["x"].shape
    step = max(1, (1 << 25) // v)
    return [(r, min(step, m - r)) for r in range(0, m, step)]


def _stats64(st):
    lse, ent = [], []
    for r, n in _chunks(st):
        _, z = _rows64(st, r, n)
        l = torch.logsumexp(z, dim=1)
        lp = z - l.unsqueeze(1)
        lse.append(l)
        ent.append(-torch.nan_to_num(torch.exp(lp) * lp, nan=0.0).sum(1))
    return torch.cat(lse), torch.cat(ent)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "logprobs":
        lse, ent = _stats64(st)
        lps, ranks, tlps, tids = [], [], [], []
        for r, n in _chunks(st):
            raw, z = _rows64(st, r, n)
            tok = st["tok"][r:r + n].long().unsqueeze(1)
            l = lse[r:r + n].unsqueeze(1)
            lps.append((z.gather(1, tok) - l).squeeze(1))
            ranks.append(1 + (raw > raw.gather(1, tok)).sum(1))
            ids = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :case["topk"]]
            tlps.append(z.gather(1, ids) - l)
            tids.append(ids)
        return (torch.cat(lps), torch.cat(ranks).to(torch.int32), lse, ent, torch.cat(tlps),
                torch.cat(tids).to(torch.int32))
    if op == "logprobs_backward":
        out = []
        for r, n in _chunks(st):
            _, z = _rows64(st, r, n)
            lse = st["lse"][r:r + n].double().unsqueeze(1)
            g = st["dlp"][r:r + n].double().unsqueeze(1)
            lp = z - lse
            p = torch.exp(lp)
            d = torch.zeros_like(p).scatter_(1, st["tok"][r:r + n].long().unsqueeze(1), 1.0)
            d = g * (d - p)
            if st["dent"] is not None:
                h = st["entropy"][r:r + n].double().unsqueeze(1)
                d -= st["dent"][r:r + n].double().unsqueeze(1) * torch.nan_to_num(p * (lp + h), nan=0.0)
            if st["temps"] is not None:
                d = d / st["temps"][r:r + n].double().unsqueeze(1)
            out.append(d)
        return torch.cat(out)
    if op == "moe_decode":
        ids, w = _route(st, torch.float64)
        x = st["x"].double()
        out = torch.zeros_like(x)
        for j in sorted(set(ids.flatten().tolist())):
            w13 = _dequant(st["w13"][0][j], st["w13"][1][j], st["w13"][2][j], torch.float64)
            h = x @ w13.t()
            gate, up = h.chunk(2, dim=1)
            a = gate * torch.sigmoid(gate) * up
            w2 = _dequant(st["w2"][0][j], st["w2"][1][j], st["w2"][2][j], torch.float64)
            weight = torch.where(ids == j, w, 0.0).sum(1, keepdim=True)
            out += weight * (a @ w2.t())
        return out, ids.to(torch.int32), w
    # int4: the sum over each group in 64 bits, then its scale
    n, k, group = case["N"], case["K"], case["group"]
    x = st["x"].double()
    y = torch.empty((case["M"], n), dtype=torch.float64, device=DEV)
    step = max(8, (1 << 25) // k // 8 * 8)
    for r in range(0, n, step):
        words = st["packed"][r:r + step].long() & 0xFFFFFFFF
        c = words.shape[0]
        q = torch.stack([(words >> (4 * b)) & 15 for b in range(8)], dim=2).view(c, k).double()
        if st["zp"] is None:
            q -= 8.0
        else:
            zw = st["zp"][r // 8:(r + c + 7) // 8].long() & 0xFFFFFFFF
            z = torch.stack([(zw >> (4 * b)) & 15 for b in range(8)], dim=1).flatten(0, 1)[:c]
            q -= z.double().repeat_interleave(group, dim=1)
        q *= st["scales"][r:r + step].double().repeat_interleave(group, dim=1)
        y[:, r:r + step] = x @ q.t()
    if st["bias"] is not None:
        y += st["bias"].double()
    return y
