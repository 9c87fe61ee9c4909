"""What is measured of the operators around a model's last block and head: the
cross entropy taken straight from hidden states and the lm_head weight with its
gradients, the gated feed-forward block with its gradients, and the 8-bit
integer product with scales for each token and channel.

``run`` computes each operator in its plain form (elementary torch operations
in float32) or, where ``own`` is true, through the library's entry points.
``exact`` computes the same outputs from the definitions in float64.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _i8(name, m, n, k, bias=False):
    return {"name": name, "op": "int8_linear", "M": m, "N": n, "K": k, "bias": bias}


def _ce(name, m, v, k, train, ignored=0.0, bias=False, dlse=False):
    return {"name": name, "op": "linear_ce", "M": m, "V": v, "K": k, "train": train, "ignored": ignored,
            "bias": bias, "dlse": dlse}


def _ffn(name, t, h, i, train):
    return {"name": name, "op": "gated_ffn", "T": t, "H": h, "I": i, "train": train}


def listed():
    return [
        # one token's logits from an int8 lm_head: the weight streams past once
        _i8("int8_1x128256x4096", 1, 128256, 4096),
        # a decode batch over the widest head
        _i8("int8_16x151936x5120", 16, 151936, 5120),
        # a ragged batch, odd vocabulary, bias
        _i8("int8_33x32003x2080", 33, 32003, 2080, True),
        # a prompt through an up projection: bound by the matrix units
        _i8("int8_4096x28672x4096", 4096, 28672, 4096),
        # scoring a prompt: the loss alone
        _ce("ce_2048x128256x4096", 2048, 128256, 4096, False),
        # a training step of the head: loss and all gradients, a few padded rows
        _ce("ce_train_4096x128256x4096", 4096, 128256, 4096, True, ignored=0.05),
        # a short answer of a small model, its prompt ignored: latency
        _ce("ce_train_17x32003x512", 17, 32003, 512, True, ignored=0.3),
        # ragged sizes, a bias, and a loss term on the lse
        _ce("ce_train_333x32003x2080", 333, 32003, 2080, True, ignored=0.1, bias=True, dlse=True),
        # one token through a dense block of the expert layer's sizes
        _ffn("ffn_1_4096x14336", 1, 4096, 14336, False),
        # a decode batch through the same block
        _ffn("ffn_16_4096x14336", 16, 4096, 14336, False),
        # a training step of the same block
        _ffn("ffn_train_4096_4096x14336", 4096, 4096, 14336, True),
        # a training step at ragged sizes
        _ffn("ffn_train_333_2080x5616", 333, 2080, 5616, True),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm, odd ones among them."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["int8_linear", "linear_ce", "gated_ffn"])
    if op == "int8_linear":
        k = 16 * _log_int(rng, 32, 512)
        n = _log_int(rng, 1000, min(152000, 151936 * 5120 // k))
        m = _log_int(rng, 1, min(4096, 4096 * 28672 * 4096 // (n * k)))
        case = _i8("", m, n, k, rng.random() < 0.3)
    elif op == "linear_ce":
        k = 16 * _log_int(rng, 32, 320)
        v = _log_int(rng, 1000, 130000)
        train = rng.random() < 0.6
        m = _log_int(rng, 1, min(4096, max(1, (4096 if train else 2048) * 128256 * 4096 // (v * k))))
        case = _ce("", m, v, k, train, rng.choice([0.0, 0.05, 0.3]), rng.random() < 0.3,
                   train and rng.random() < 0.3)
    else:
        h = 16 * _log_int(rng, 32, 320)
        i = 16 * _log_int(rng, 32, 896)
        train = rng.random() < 0.5
        t = _log_int(rng, 1, min(4096, max(1, 4096 * 4096 * 14336 // (h * i))))
        case = _ffn("", t, h, i, train)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, std, g):
    """bf16 normal values, made in pieces of rows."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    rows = max(1, (1 << 26) // shape[1])
    for r in range(0, shape[0], rows):
        n = min(rows, shape[0] - r)
        out[r:r + n] = (std * torch.randn((n, shape[1]), generator=g, device=DEV)).to(torch.bfloat16)
    return out


def _int8_rows(w):
    """A weight kept as int8: one scale per channel, made once when it is loaded."""
    q = torch.empty(w.shape, dtype=torch.int8, device=DEV)
    s = torch.empty((w.shape[0],), dtype=torch.float32, device=DEV)
    rows = max(1, (1 << 26) // w.shape[1])
    for r in range(0, w.shape[0], rows):
        f = w[r:r + rows].float()
        c = (f.abs().amax(1) / 127.0).clamp_min(1e-12)
        s[r:r + rows] = c
        q[r:r + rows] = torch.round(f / c.unsqueeze(1)).clamp_(-127, 127).to(torch.int8)
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "int8_linear":
        m, n, k = case["M"], case["N"], case["K"]
        st["wq"], st["ws"] = _int8_rows(_normal((n, k), 0.02, g))
        # normed hidden states: a broad bulk, some channels larger in every token
        ch = torch.where(torch.rand((k,), generator=g, device=DEV) < 0.01, 8.0, 1.0)
        st["x"] = (torch.randn((m, k), generator=g, device=DEV) * ch).to(torch.bfloat16)
        st["bias"] = _normal((1, n), 0.5, g)[0] if case["bias"] else None
    elif op == "linear_ce":
        m, v, k = case["M"], case["V"], case["K"]
        w = _normal((v, k), 0.02 * math.sqrt(4096 / k), g)
        tok = torch.randint(0, v, (m,), generator=g, device=DEV)
        x = torch.randn((m, k), generator=g, device=DEV)
        # most targets are likely ones: the hidden state leans towards their row
        lean = torch.where(torch.rand((m, 1), generator=g, device=DEV) < 0.7, 8.0, 0.0)
        row = w[tok].float()
        x += lean * row / row.norm(dim=1, keepdim=True)
        st["x"], st["w"] = x.to(torch.bfloat16), w
        gone = torch.rand((m,), generator=g, device=DEV) < case["ignored"]
        gone[m - 1] = False
        st["tok"] = torch.where(gone, -100, tok).to(torch.int32)
        st["bias"] = _normal((1, v), 0.5, g)[0] if case["bias"] else None
        if case["train"]:
            # a mean over the rows that count, some rows weighted, and its loss scale
            scale = 1.0 / (~gone).sum()
            st["dloss"] = scale * (0.5 + torch.rand((m,), generator=g, device=DEV))
            st["dlse"] = 0.01 * scale * torch.randn((m,), generator=g, device=DEV) if case["dlse"] else None
    else:
        t, h, i = case["T"], case["H"], case["I"]
        st["x"] = _normal((t, h), 1.0, g)
        st["w13"] = _normal((2 * i, h), 1.3 / math.sqrt(h), g)
        st["w2"] = _normal((h, i), 1.0 / math.sqrt(i), g)
        if case["train"]:
            st["dy"] = _normal((t, h), 1.0 / math.sqrt(t * h), g)
    if own:
        # the workspace that a program keeps
        from nvfp4_w4a16_lm_amd import binding as B
        if op == "linear_ce":
            st["ws"] = B.linear_ce_workspace(case["M"], case["V"], case["K"], DEV, backward=case["train"])
        elif op == "gated_ffn":
            st["ws"] = B.gated_ffn_workspace(case["T"], case["H"], case["I"], DEV, backward=case["train"])
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _run_own(st):
    from nvfp4_w4a16_lm_amd import binding as B
    case = st["case"]
    op = case["op"]
    if op == "int8_linear":
        xq, xs = B.nvfp4_int8_quantize_rows(st["x"])
        return B.nvfp4_int8_gemm(xq, xs, st["wq"], st["ws"], bias=st["bias"])
    if op == "linear_ce":
        r = B.nvfp4_linear_ce(st["x"], st["w"], st["tok"], bias=st["bias"], workspace=st["ws"])
        if not case["train"]:
            return r.loss, r.lse
        dx, dw, db = B.nvfp4_linear_ce_backward(st["x"], st["w"], st["tok"], r.stats, st["dloss"], bias=st["bias"],
                                                dlse=st["dlse"], workspace=st["ws"])
        return (r.loss, r.lse, dx, dw) + (() if db is None else (db,))
    if not case["train"]:
        return B.nvfp4_gated_ffn(st["x"], st["w13"], st["w2"], workspace=st["ws"])
    y, h = B.nvfp4_gated_ffn(st["x"], st["w13"], st["w2"], keep_h=True, workspace=st["ws"])
    return (y,) + B.nvfp4_gated_ffn_backward(st["x"], h, st["w13"], st["w2"], st["dy"], workspace=st["ws"])


def _plain_int8(st):
    x = st["x"].float()
    s = (x.abs().amax(1, keepdim=True) / 127.0).clamp_min(1e-12)
    q = torch.round(x / s).clamp_(-127, 127)
    y = (q @ st["wq"].float().t()) * s * st["ws"]
    if st["bias"] is not None:
        y += st["bias"].float()
    return y.to(torch.bfloat16)


def _plain_ce(st):
    case = st["case"]
    keep = st["tok"] >= 0
    tok = st["tok"].clamp_min(0).long().unsqueeze(1)
    x, w = st["x"].float(), st["w"].float()
    z = x @ w.t()
    if st["bias"] is not None:
        z += st["bias"].float()
    top = z.amax(1, keepdim=True)
    zt = z.gather(1, tok)
    e = torch.exp(z.sub_(top))
    s = e.sum(1, keepdim=True)
    lse = (top + torch.log(s)).squeeze(1)
    loss = ((top - zt) + torch.log(s)).squeeze(1)
    loss, lse = torch.where(keep, loss, 0.0), torch.where(keep, lse, 0.0)
    if not case["train"]:
        return loss, lse
    d = torch.where(keep, st["dloss"], 0.0).unsqueeze(1)
    c = d if st["dlse"] is None else d + torch.where(keep, st["dlse"], 0.0).unsqueeze(1)
    e *= c / s
    e.scatter_add_(1, tok, -d)
    out = (loss, lse, (e @ w).to(torch.bfloat16), (e.t() @ x).to(torch.bfloat16))
    return out if st["bias"] is None else out + (e.sum(0).to(torch.bfloat16),)


def _plain_ffn(st):
    case = st["case"]
    i = case["I"]
    x, w13, w2 = st["x"].float(), st["w13"].float(), st["w2"].float()
    h = x @ w13.t()
    g, u = h[:, :i], h[:, i:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    a = g * sig * u
    y = (a @ w2.t()).to(torch.bfloat16)
    if not case["train"]:
        return y
    dy = st["dy"].float()
    da = dy @ w2
    dh = torch.cat((da * u * sig * (1.0 + g * (1.0 - sig)), da * g * sig), 1)
    return (y, (dh @ w13).to(torch.bfloat16), (dh.t() @ x).to(torch.bfloat16), (dy.t() @ a).to(torch.bfloat16))


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "int8_linear":
        return _plain_int8(state)
    return _plain_ce(state) if op == "linear_ce" else _plain_ffn(state)


# ---------------------------------------------------------------------------
# Work, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "int8_linear":
        m, n, k = case["M"], case["N"], case["K"]
        return {"bytes": n * k + 2 * m * k + 2 * m * n + 4 * n + (2 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if op == "linear_ce":
        m, v, k = case["M"], case["V"], case["K"]
        rows = m * (1.0 - case["ignored"])               # what counts, on average
        b = 2 * (m + v) * k + 12 * m + (2 * v if case["bias"] else 0)
        if not case["train"]:
            return {"bytes": b, "flops": int(2 * rows * v * k)}
        # the logits, the logits again (they are not kept) and the two gradients' products
        return {"bytes": b + 2 * (m + v) * k + (2 * v if case["bias"] else 0) + 8 * m,
                "flops": int(8 * rows * v * k)}
    t, h, i = case["T"], case["H"], case["I"]
    if not case["train"]:
        return {"bytes": 6 * h * i + 4 * t * h, "flops": 6 * t * h * i}
    return {"bytes": 12 * h * i + 8 * t * h, "flops": 18 * t * h * i}


def _exact_int8(st):
    # codes from the ratio 127 x / amax, which float64 places on the right side of every border
    x = st["x"].double()
    top = x.abs().amax(1, keepdim=True)
    s = torch.clamp(top / 127.0, min=1e-12)
    q = torch.round(torch.where(s > 1e-12, x * 127.0 / top.clamp_min(1e-300), x / s))
    y = torch.empty((x.shape[0], st["wq"].shape[0]), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 27) // x.shape[1])
    for r in range(0, y.shape[1], step):
        w = st["wq"][r:r + step].double() * st["ws"][r:r + step].double().unsqueeze(1)
        y[:, r:r + step] = (q * s) @ w.t()
    if st["bias"] is not None:
        y += st["bias"].double()
    return y


def _exact_ce(st):
    case = st["case"]
    m, v = case["M"], case["V"]
    rows = torch.nonzero(st["tok"] >= 0).flatten()       # only the rows that count
    tok = st["tok"][rows].long()
    x = st["x"][rows].double()
    step = max(1, (1 << 27) // max(rows.numel(), case["K"]))

    def logits(r):
        z = x @ st["w"][r:r + step].double().t()
        return z if st["bias"] is None else z + st["bias"][r:r + step].double()

    lse = torch.full((rows.numel(),), -math.inf, dtype=torch.float64, device=DEV)
    zt = torch.zeros_like(lse)
    for r in range(0, v, step):
        z = logits(r)
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        here = (tok >= r) & (tok < r + step)
        zt[here] = z[here, tok[here] - r]

    def whole(t):
        return torch.zeros((m,) + t.shape[1:], dtype=torch.float64, device=DEV).index_copy_(0, rows, t)

    out = (whole(lse - zt), whole(lse))
    if not case["train"]:
        return out
    d = st["dloss"][rows].double().unsqueeze(1)
    e = 0.0 if st["dlse"] is None else st["dlse"][rows].double().unsqueeze(1)
    dx = torch.zeros_like(x)
    dw = torch.empty(st["w"].shape, dtype=torch.float64, device=DEV)
    db = torch.empty((v,), dtype=torch.float64, device=DEV)
    for r in range(0, v, step):
        p = torch.exp(logits(r) - lse.unsqueeze(1))
        one = torch.arange(r, r + p.shape[1], device=DEV).unsqueeze(0) == tok.unsqueeze(1)
        dz = d * (p - one.double()) + e * p
        dx += dz @ st["w"][r:r + step].double()
        dw[r:r + step] = dz.t() @ x
        db[r:r + step] = dz.sum(0)
    out += (whole(dx), dw)
    return out if st["bias"] is None else out + (db,)


def _exact_ffn(st):
    case = st["case"]
    t, h, i = case["T"], case["H"], case["I"]
    x, w13, w2 = st["x"].double(), st["w13"].double(), st["w2"].double()
    g, u = x @ w13[:i].t(), x @ w13[i:].t()
    sig = torch.sigmoid(g)
    a = g * sig * u
    y = a @ w2.t()
    if not case["train"]:
        return y
    dy = st["dy"].double()
    da = dy @ w2
    du = da * g * sig
    dg = da * u * (sig + g * sig * torch.sigmoid(-g))
    dx = dg @ w13[:i] + du @ w13[i:]
    return y, dx, torch.cat((dg.t() @ x, du.t() @ x)), dy.t() @ a


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "int8_linear":
        return _exact_int8(st)
    return _exact_ce(st) if case["op"] == "linear_ce" else _exact_ffn(st)
