"""GPU parity of the gated feed-forward block and its gradients with the float64
oracle: sizes around every tile width, single tokens, saturated gates,
differences, outputs written exactly, graph replays and given streams."""

import numpy as np
import pytest
import torch

import oracle.dense_oracle as D
from nvfp4_w4a16_lm_amd import binding as B

from gpu_util import DEV
from test_gpu_graphs import capture

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def bf16(rng, *shape, sigma=1.0):
    return torch.from_numpy(sigma * rng.standard_normal(shape)).to(BF16)


def make(t, h, i, seed, gate=1.3):
    rng = np.random.default_rng(seed)
    return [bf16(rng, t, h), bf16(rng, 2 * i, h, sigma=gate / np.sqrt(h)), bf16(rng, h, i, sigma=1 / np.sqrt(i)),
            bf16(rng, t, h, sigma=0.1)]


def f64(t):
    return t.cpu().double().numpy()


def within(got, want, bound, what):
    err = np.abs(f64(got) - want)
    assert np.all(err <= bound), (what, err.max(), (err / bound).max())


def check(t, h, i, seed, gate=1.3):
    a = make(t, h, i, seed, gate)
    x, w13, w2, dy = (v.to(DEV) for v in a)
    y, kept = B.nvfp4_gated_ffn(x, w13, w2, keep_h=True)
    (wy, wh, wa), (by, bh, ba) = D.gated_ffn(*map(f64, a[:3]))
    within(y, wy, by, "y")
    within(kept.h, wh, bh, "h")
    within(kept.act, wa, ba, "act")
    assert torch.equal(y, B.nvfp4_gated_ffn(x, w13, w2))
    grads = B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dy)
    want, bounds = D.gated_ffn_backward(f64(x), f64(kept.h), f64(kept.act), f64(w13), f64(w2), f64(dy))
    for g, v, b, what in zip(grads, want, bounds, ("dx", "dw13", "dw2")):
        within(g, v, b, what)
    return (x, w13, w2, dy), kept, grads


@pytest.mark.parametrize("t,h,i", [
    (1, 16, 16), (1, 528, 1040), (2, 64, 48), (3, 256, 128), (7, 272, 528), (15, 1040, 144), (16, 512, 256), (17, 144, 272),
    (31, 80, 400), (32, 256, 256), (33, 528, 112), (64, 336, 640), (65, 272, 528), (128, 144, 144), (129, 528, 272),
    (200, 528, 1040), (257, 144, 528), (333, 2080, 560), (600, 272, 272)])
def test_sizes(t, h, i):
    check(t, h, i, seed=t + h + i)


@pytest.mark.parametrize("t,h,i", [(333, 208, 11008), (333, 208, 22016), (700, 528, 8208), (1100, 2080, 2064), (450, 2080, 5616)])
def test_wide_tiles(t, h, i):
    """Sizes at which the widest tiles are taken: 192 and 256 rows, 256 of the weights' gradients."""
    check(t, h, i, seed=t + i)


@pytest.mark.parametrize("t", [1, 16, 100])
def test_saturated_gates(t):
    """Gates of hundreds: the logistic function at 0 and 1, its exponential at infinity."""
    check(t, 64, 128, seed=t, gate=150.0)


def test_long_rows():
    check(1, 4096, 2048, seed=1)
    check(12, 1024, 8192, seed=2)


def test_gradient_against_differences():
    a = make(20, 64, 96, seed=3)
    n = [f64(v) for v in a]
    (x, w13, w2, dy), kept, grads = check(20, 64, 96, seed=3)
    # kept values are a little off between the passes: h by its sums, a by its rounding too
    (_, h, act), (_, bh, ba) = D.gated_ffn(*n[:3])
    i = 96
    g, u, da, s = h[:, :i], h[:, i:], np.abs(n[3] @ n[2]), D.sigmoid(h[:, :i])
    eg, eu = bh[:, :i], bh[:, i:]                        # |silu'| <= 1.1, |silu''| <= 0.5
    e = 1.1 * np.concatenate((da * (1.1 * eu + 0.5 * np.abs(u) * eg), da * 1.1 * eg), 1)
    extra = (e @ np.abs(n[1]), e.T @ np.abs(n[0]), np.abs(n[3]).T @ ba)
    _, bounds = D.gated_ffn_backward(n[0], f64(kept.h), f64(kept.act), n[1], n[2], n[3])
    rng = np.random.default_rng(1)
    f = lambda *p: (D.gated_ffn(*p)[0][0] * n[3]).sum()
    for which, grad in enumerate(grads):
        d = rng.standard_normal(n[which].shape)
        up, down = n[:3], n[:3]
        up[which], down[which] = n[which] + 1e-5 * d, n[which] - 1e-5 * d
        diff = (f(*up) - f(*down)) / 2e-5
        assert abs(diff - (f64(grad) * d).sum()) <= ((bounds[which] + extra[which]) * np.abs(d)).sum() + 1e-5


def test_infinite_and_nan_rows_stay_alone():
    x, w13, w2, dy = (v.to(DEV) for v in make(40, 64, 96, seed=5))
    x[3, 5], x[7, 9] = float("nan"), float("inf")
    y, h = B.nvfp4_gated_ffn(x, w13, w2, keep_h=True)
    bad = torch.zeros(40, dtype=torch.bool, device=DEV)
    bad[[3, 7]] = True
    assert torch.isfinite(y[~bad]).all() and not torch.isfinite(y[3]).any()
    dx, _, _ = B.nvfp4_gated_ffn_backward(x, h, w13, w2, dy)
    assert torch.isfinite(dx[~bad]).all()


@pytest.mark.parametrize("t", [1, 15, 16, 17, 40])
def test_infinite_weights_of_the_down_projection(t):
    """An infinity in w2 makes its column infinite with the activation's sign, whether the activation enters as a pair
    or rounded; two of opposite signs make it NaN; the other columns are what they were."""
    h, i = 64, 1040
    n = make(t, h, i, seed=11)
    n[2][5, 3], n[2][9, 1000], n[2][40, 7], n[2][63, 0] = float("inf"), -float("inf"), float("inf"), float("nan")
    n[2][40, 8] = float("inf")
    x, w13, w2, _ = (v.to(DEV) for v in n)
    y = f64(B.nvfp4_gated_ffn(x, w13, w2))
    (_, _, a), (_, _, ba) = D.gated_ffn(f64(n[0]), f64(n[1]), np.zeros((h, i)))
    assert np.all(np.abs(a[:, [3, 7, 8, 1000]]) > ba[:, [3, 7, 8, 1000]])           # their signs are sure
    sign = np.sign(a)
    assert np.array_equal(y[:, 5], sign[:, 3] * np.inf) and np.array_equal(y[:, 9], -sign[:, 1000] * np.inf)
    want = np.where(sign[:, 7] == sign[:, 8], sign[:, 7] * np.inf, np.nan)
    assert np.array_equal(y[:, 40], want, equal_nan=True) and np.isnan(y[:, 63]).all()
    rest = np.setdiff1d(np.arange(h), [5, 9, 40, 63])
    w2 = f64(n[2]).copy()
    w2[[5, 9, 40, 63]] = 0.0
    (wy, _, _), (by, _, _) = D.gated_ffn(f64(n[0]), f64(n[1]), w2)
    assert np.all(np.abs(y[:, rest] - wy[:, rest]) <= by[:, rest])


@pytest.mark.parametrize("t", [1, 20, 150])
def test_buffers_are_written_exactly(t):
    lib = B.load_library()
    h, i = 80, 112
    x, w13, w2, dy = (v.to(DEV) for v in make(t, h, i, seed=6))
    y, kept = B.nvfp4_gated_ffn(x, w13, w2, keep_h=True)
    want = B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dy)
    size = int(lib.nvfp4_gated_ffn_workspace_bytes(t, h, i, 1))
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    outs = [torch.full((n + 32,), 3.0, dtype=dt, device=DEV)
            for n, dt in ((t * h, BF16), (2 * t * i, torch.float32), (t * i, BF16), (t * h, BF16), (2 * i * h, BF16),
                          (h * i, BF16))]
    p = [o.data_ptr() for o in outs]
    s = torch.cuda.current_stream().cuda_stream
    xp, w13p, w2p, dyp = (v.data_ptr() for v in (x, w13, w2, dy))
    assert lib.nvfp4_gated_ffn(xp, t, h, w13p, w2p, i, p[1], p[2], ws.data_ptr(), p[0], s) == 0
    assert lib.nvfp4_gated_ffn_backward(xp, t, h, p[1], p[2], w13p, w2p, i, dyp, ws.data_ptr(), *p[3:], s) == 0
    torch.cuda.synchronize()
    for got, ref in zip(outs, (y, *kept, *want)):
        assert torch.equal(got[:ref.numel()], ref.flatten()) and torch.all(got[ref.numel():] == 3.0)
    assert torch.all(ws[size:] == 0xFF)
    for keep in range(3):                                # each gradient alone
        alone = [torch.full_like(o, 3.0) for o in outs[3:]]
        a = [o.data_ptr() if j == keep else None for j, o in enumerate(alone)]
        assert lib.nvfp4_gated_ffn_backward(xp, t, h, p[1], p[2], w13p, w2p, i, dyp, ws.data_ptr(), *a, s) == 0
        torch.cuda.synchronize()
        for j, o in enumerate(alone):
            assert torch.equal(o, outs[3 + j]) if j == keep else torch.all(o == 3.0)


@pytest.mark.parametrize("t", [1, 16, 100, 300])
def test_graph_replays(t):
    h, i = 272, 528
    x, w13, w2, dy = (v.to(DEV) for v in make(t, h, i, seed=7))
    ws = B.gated_ffn_workspace(t, h, i, DEV)
    held = []

    def call():
        y, kept = B.nvfp4_gated_ffn(x, w13, w2, keep_h=True, workspace=ws)
        return (y, *kept, *B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dy, workspace=ws))
    graph = capture(lambda: held.append(call()))
    rng = np.random.default_rng(t)
    for _ in range(3):
        x.copy_(bf16(rng, t, h))
        dy.copy_(bf16(rng, t, h))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in held[-1]]
        for a, b in zip(got, call()):
            assert torch.equal(a, b)


def test_given_stream_with_wide_input():
    x, w13, w2, dy = (v.to(DEV) for v in make(20, 144, 272, seed=8))
    y, kept = B.nvfp4_gated_ffn(x, w13, w2, keep_h=True)
    want = B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dy)
    wide = lambda v: torch.stack([v, v], -1)[..., 0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y2, h2 = B.nvfp4_gated_ffn(wide(x), wide(w13), wide(w2), keep_h=True, stream=side)
    g2 = B.nvfp4_gated_ffn_backward(wide(x), h2, wide(w13), wide(w2), wide(dy), stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, *kept, *want), (y2, *h2, *g2)))


def test_workspace_kept_for_the_largest_batch():
    """One workspace of the largest batch, for every smaller one: the results are those of a fresh one."""
    h, i = 144, 1040
    x, w13, w2, dy = (v.to(DEV) for v in make(1025, h, i, seed=10))
    ws = B.gated_ffn_workspace(1025, h, i, DEV)
    for t in (1025, 1024, 513, 257, 256, 129, 128, 65, 33, 32, 17, 16, 1):
        y, kept = B.nvfp4_gated_ffn(x[:t], w13, w2, keep_h=True)
        want = (y, *kept, *B.nvfp4_gated_ffn_backward(x[:t], kept, w13, w2, dy[:t]))
        y, kept = B.nvfp4_gated_ffn(x[:t], w13, w2, keep_h=True, workspace=ws)
        got = (y, *kept, *B.nvfp4_gated_ffn_backward(x[:t], kept, w13, w2, dy[:t], workspace=ws))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), t


@pytest.mark.parametrize("t", [1, 40])
def test_gradients_left_out_and_given_buffers(t):
    """Every choice of gradients through the binding: those left out are None, the others are what they are together,
    made or in the caller's buffers; of an empty batch a buffer becomes zero."""
    x, w13, w2, dy = (v.to(DEV) for v in make(t, 80, 112, seed=12))
    _, kept = B.nvfp4_gated_ffn(x, w13, w2, keep_h=True)
    want = B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dy)
    names = ("dx", "dw13", "dw2")
    for mask in range(8):
        got = B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dy, **{n: bool(mask >> j & 1) for j, n in enumerate(names)})
        assert all(torch.equal(g, w) if mask >> j & 1 else g is None for j, (g, w) in enumerate(zip(got, want)))
    bufs = [torch.full_like(v, 3.0) for v in want]
    got = B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dy, **dict(zip(names, bufs)))
    assert all(g is b and torch.equal(g, w) for g, b, w in zip(got, bufs, want))
    none = B.GatedKept(kept.h[:0], kept.act[:0])
    dx, d13, d2 = B.nvfp4_gated_ffn_backward(x[:0], none, w13, w2, dy[:0], dw13=bufs[1].fill_(3.0), dw2=False)
    assert dx.shape == (0, 80) and d13 is bufs[1] and not d13.any() and d2 is None
    for bad in (dict(dx=bufs[0][:-1].T), dict(dw13=bufs[1].float()), dict(dw2=bufs[2].cpu())):
        with pytest.raises(ValueError):
            B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dy, **bad)


def test_empty_batch_and_refusals():
    x, w13, w2, dy = (v.to(DEV) for v in make(4, 32, 48, seed=9))
    y, kept = B.nvfp4_gated_ffn(x[:0], w13, w2, keep_h=True)
    assert y.shape == (0, 32) and kept.h.shape == (0, 96) and kept.act.shape == (0, 48)
    dx, d13, d2 = B.nvfp4_gated_ffn_backward(x[:0], kept, w13, w2, dy[:0])
    assert dx.shape == (0, 32) and not d13.any() and not d2.any()
    y, kept = B.nvfp4_gated_ffn(x, w13, w2, keep_h=True)
    for bad in ((x, w13[:95], w2), (x, w13, w2[:31]), (x[:, :16].contiguous(), w13, w2)):
        with pytest.raises(ValueError):
            B.nvfp4_gated_ffn(*bad)
    with pytest.raises(ValueError):
        B.nvfp4_gated_ffn_backward(x, B.GatedKept(kept.h.to(BF16), kept.act), w13, w2, dy)
    with pytest.raises(ValueError):
        B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dy[:3])
    with pytest.raises(ValueError):
        B.nvfp4_gated_ffn(x, w13, w2, workspace=torch.empty((16,), dtype=torch.uint8, device=DEV))
