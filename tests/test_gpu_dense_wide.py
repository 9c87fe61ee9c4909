"""Tensors of more than 2^31 elements, and weights of nearly 2^32 bytes, through the
int8, cross entropy and gated calls, against the float64 oracle.

The oracle sees only what counts: tokens outside a few hundred are masked by a bias
of -inf, rows outside them have no gradient coming in, units outside them have
zero weights.  All of that is exact (probability 0, dz 0, activation 0), so that
the rest is the oracle's result on the few, and what lies outside must be exactly
0.  The few lie at both ends and around the 2^31st element."""

import numpy as np
import pytest
import torch

import oracle.dense_oracle as D
from nvfp4_w4a16_lm_amd import binding as B

from gpu_util import DEV

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(shape, g, sigma=1.0):
    return torch.empty(shape, dtype=BF16, device=DEV).normal_(0.0, sigma, generator=g)


def few(n, width, seed):
    """Sorted indices: both ends, around the row that holds element 2^31 of rows of `width`, and some between, in runs:
    sums over them then round about once for four of them, as the oracle counts."""
    rng = np.random.default_rng(seed)
    at = 2 ** 31 // width
    near = np.arange(at - 20, min(at + 20, n)) if 20 < at < n else np.arange(0)
    runs = (8 * rng.integers(0, n // 8, 15))[:, None] + np.arange(8)
    return np.unique(np.concatenate((np.arange(20), np.arange(n - 20, n), near, runs.flatten())))


def f64(t):
    return t.cpu().double().numpy()


def within(got, want, bound, what):
    got = f64(got)
    both = np.isfinite(want)
    assert np.array_equal(got[~both], want[~both], equal_nan=True), what
    err = np.abs(got[both] - want[both])
    assert np.all(err <= bound[both]), (what, err.max(), (err / bound[both]).max())


def all_zero_but(t, rows, dim=0):
    """t is zero outside `rows` of a dimension."""
    n = torch.zeros((t.shape[dim],), dtype=torch.int64, device=DEV)
    step = max(1, (1 << 28) // t.shape[1])
    for r in range(0, t.shape[0], step):
        part = t[r:r + step] != 0
        if dim == 0:
            n[r:r + step] = part.sum(1)
        else:
            n += part.sum(0)
    n[torch.from_numpy(rows).to(DEV)] = 0
    assert not n.any()


@pytest.mark.parametrize("m", [3, 70, 300])
def test_int8_weight(m):
    n, k = 524309, 4112
    g = gen(m)
    a = normal((n, k), g, 0.02)
    wq, ws = B.nvfp4_int8_quantize_rows(a)
    rows = few(n, k, m)
    idx = torch.from_numpy(rows).to(DEV)
    cq, cs = D.int8_quantize_rows(f64(a[idx]))
    assert np.array_equal(wq[idx].cpu().numpy(), cq) and np.array_equal(ws[idx].cpu().numpy(), cs)
    del a
    xq = torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int8, device=DEV)
    xs = torch.full((m,), 0.01, device=DEV)
    y = B.nvfp4_int8_gemm(xq, xs, wq, ws)
    want, bound = D.int8_gemm(xq.cpu().numpy(), xs.cpu().numpy(), cq, cs)
    within(y[:, idx], want, bound, "y")


def test_int8_output():
    m, n, k = 40009, 65537, 32
    g = gen(1)
    xq, wq = (torch.randint(-128, 128, (r, k), generator=g, dtype=torch.int8, device=DEV) for r in (m, n))
    xs, ws = (0.01 + 0.01 * torch.rand((r,), generator=g, device=DEV) for r in (m, n))
    y = B.nvfp4_int8_gemm(xq, xs, wq, ws)
    rows = few(m, n, 1)
    idx = torch.from_numpy(rows).to(DEV)
    want, bound = D.int8_gemm(xq[idx].cpu().numpy(), xs[idx].cpu().numpy(), wq.cpu().numpy(), ws.cpu().numpy())
    within(y[idx], want, bound, "y")


@pytest.mark.parametrize("m", [5, 150, 600])
def test_cross_entropy_weight(m):
    """A vocabulary of 524309 rows of 4112."""
    v, k = 524309, 4112
    g = gen(m)
    w = normal((v, k), g, 1.3 / k ** 0.5)
    live = few(v, k, m)
    idx = torch.from_numpy(live).to(DEV)
    bias = torch.full((v,), -float("inf"), dtype=BF16, device=DEV)
    bias[idx] = normal((len(live),), g)
    rng = np.random.default_rng(m)
    at = rng.integers(0, len(live), m)
    x = normal((m, k), g)
    t = torch.from_numpy(live[at].astype(np.int32)).to(DEV)
    dloss = torch.from_numpy(rng.standard_normal(m).astype(np.float32)).to(DEV)
    r = B.nvfp4_linear_ce(x, w, t, bias=bias)
    dx, dw, db = B.nvfp4_linear_ce_backward(x, w, t, r.stats, dloss, bias=bias)
    nx, nw, nb, nd = f64(x), f64(w[idx]), f64(bias[idx]), f64(dloss)
    loss, lse, bl, be = D.linear_ce(nx, nw, at, nb)
    within(r.loss, loss, bl, "loss")
    within(r.lse, lse, be, "lse")
    want, bounds = D.linear_ce_backward(nx, nw, at, nd, None, nb)
    within(dx, want[0], bounds[0], "dx")
    within(dw[idx], want[1], bounds[1], "dw")
    within(db[idx], want[2], bounds[2], "db")
    all_zero_but(dw, live)
    all_zero_but(db.unsqueeze(1), live)


@pytest.mark.parametrize("m,v,k", [(131101, 40, 16400), (40009, 65537, 16)])
def test_cross_entropy_rows(m, v, k):
    """Hidden states, and logits, of more than 2^31 elements; every row counts, few have a gradient coming in."""
    g = gen(v)
    x, w = normal((m, k), g), normal((v, k), g, 1.3 / k ** 0.5)
    t = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    rows = few(m, max(k, v), v)
    idx = torch.from_numpy(rows).to(DEV)
    dloss = torch.zeros((m,), device=DEV)
    dloss[idx] = torch.randn((len(rows),), generator=g, device=DEV)
    r = B.nvfp4_linear_ce(x, w, t)
    dx, dw, _ = B.nvfp4_linear_ce_backward(x, w, t, r.stats, dloss)
    nx, nw, nt, nd = f64(x[idx]), f64(w), t[idx].cpu().numpy().astype(np.int64), f64(dloss[idx])
    loss, lse, bl, be = D.linear_ce(nx, nw, nt)
    within(r.loss[idx], loss, bl, "loss")
    within(r.lse[idx], lse, be, "lse")
    want, bounds = D.linear_ce_backward(nx, nw, nt, nd)
    within(dx[idx], want[0], bounds[0], "dx")
    within(dw, want[1], bounds[1], "dw")
    all_zero_but(dx, rows)


def check_gated(t, h, i, rows, units):
    """Units outside `units` have zero rows in w13, rows outside `rows` no gradient."""
    g = gen(t)
    x = normal((t, h), g)
    w13 = torch.zeros((2 * i, h), dtype=BF16, device=DEV)
    both = torch.from_numpy(np.concatenate((units, units + i))).to(DEV)
    w13[both] = normal((2 * len(units), h), g, 1.3 / h ** 0.5)
    w2 = normal((h, i), g, len(units) ** -0.5)
    dy = torch.zeros((t, h), dtype=BF16, device=DEV)
    idx = torch.from_numpy(rows).to(DEV)
    dy[idx] = normal((len(rows), h), g, 0.1)
    y, kept = B.nvfp4_gated_ffn(x, w13, w2, keep_h=True)
    dx, dw13, dw2 = B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dy)
    u = both[:len(units)]
    nx, n13, n2, nd = f64(x[idx]), f64(w13[both]), f64(w2[:, u]), f64(dy[idx])
    pair = nx if t <= 16 else np.concatenate((nx, np.zeros((max(0, 17 - len(rows)), h))))   # the oracle goes by the tokens
    (wy, wh, wa), (by, bh, ba) = D.gated_ffn(pair, n13, n2)
    n = len(rows)
    within(y[idx], wy[:n], by[:n], "y")
    within(kept.h[idx][:, both], wh[:n], bh[:n], "h")
    within(kept.act[idx][:, u], wa[:n], ba[:n], "act")
    want, bounds = D.gated_ffn_backward(nx, f64(kept.h[idx][:, both]), f64(kept.act[idx][:, u]), n13, n2, nd)
    within(dx[idx], want[0], bounds[0], "dx")
    within(dw13[both], want[1], bounds[1], "dw13")
    within(dw2[:, u], want[2], bounds[2], "dw2")
    all_zero_but(kept.act, units, dim=1)
    all_zero_but(dx, rows)
    all_zero_but(dw13, both.cpu().numpy())
    all_zero_but(dw2, units, dim=1)


@pytest.mark.parametrize("t", [3, 70, 300])
def test_gated_weights(t):
    """The most that is accepted: I * H = 0x38000000."""
    check_gated(t, 32768, 28672, np.arange(t), few(28672, 1 << 40, t))


def test_gated_projections():
    check_gated(131101, 48, 8208, few(131101, 2 * 8208, 1), np.arange(8208))
