"""GPU parity of the int8 row quantizer and product with their oracle: every
code, scales, exact sums of the extreme codes, odd sizes around every tile
width, bias, outputs written exactly, graph replays and given streams."""

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


def check_quant(a):
    q, s = B.nvfp4_int8_quantize_rows(a.to(DEV))
    torch.cuda.synchronize()
    wq, ws = D.int8_quantize_rows(a.double().numpy())
    assert np.array_equal(s.cpu().numpy(), ws)
    bad = np.argwhere(q.cpu().numpy() != wq)
    assert len(bad) == 0, (bad[:4], a[bad[0][0], bad[0][1]], q[bad[0][0], bad[0][1]], wq[bad[0][0], bad[0][1]])


@pytest.mark.parametrize("r,k", [(1, 16), (3, 48), (7, 528), (2, 8192), (3, 8208), (2, 20016)])
def test_quantizer_sizes(r, k):
    check_quant(bf16(np.random.default_rng(r + k), r, k, sigma=3.0))


def test_quantizer_special_rows():
    k = 512
    rng = np.random.default_rng(5)
    grid = torch.from_numpy(rng.integers(-255, 256, (12, k)).astype(np.float64))      # borders are hit often
    rows = torch.zeros((22, k), dtype=torch.float64)
    rows[:12] = grid * torch.tensor([2.0 ** e for e in range(-6, 6)]).unsqueeze(1)
    for i, top in enumerate((127.0, 254.0, 128.0, 255.0, 1.0)):
        rows[12 + i] = torch.from_numpy(rng.integers(-127, 128, k)) * top / 254.0
        rows[12 + i, 7] = -top
    rows[17] = 0.0
    rows[18, 3] = 2.0 ** -133                                                         # the least bf16
    rows[19] = torch.from_numpy(rng.uniform(-1, 1, k)) * 3.3e38
    rows[20] = torch.from_numpy(rng.uniform(-1, 1, k)) * 1e-10                        # scale 1e-12
    rows[21] = torch.from_numpy(rng.uniform(-1, 1, k)) * 1.4e-10
    check_quant(rows.to(BF16))


@pytest.mark.parametrize("k", [16, 528, 8208, 20016])
@pytest.mark.parametrize("bad", [float("nan"), -float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_finite_stay_so(k, bad):
    """A NaN or an infinity anywhere in a row: scale NaN, codes 0, and all its products NaN, as a row of x and as
    a row of the weight; the other rows as without it."""
    rng = np.random.default_rng(k)
    a = bf16(rng, 40, k)
    want = [t.clone() for t in B.nvfp4_int8_quantize_rows(a.to(DEV))]
    rows = {0: 0, 7: k - 1, 20: k // 2, 39: min(k - 1, 8195)}
    for row, at in rows.items():
        a[row, at] = bad
    q, s = B.nvfp4_int8_quantize_rows(a.to(DEV))
    wq, ws = D.int8_quantize_rows(a.double().numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    gone = torch.zeros(40, dtype=torch.bool, device=DEV)
    gone[list(rows)] = True
    assert torch.isnan(s[gone]).all() and not q[gone].any()
    assert torch.equal(q[~gone], want[0][~gone]) and torch.equal(s[~gone], want[1][~gone])
    other = codes(rng, 33, k).to(DEV)
    one = torch.full((33,), 0.01, device=DEV)
    bias = bf16(rng, 33).to(DEV)
    y = B.nvfp4_int8_gemm(q, s, other, one, bias)
    assert torch.isnan(y[gone]).all() and torch.isfinite(y[~gone]).all()
    y = B.nvfp4_int8_gemm(other, one, q, s)
    assert torch.isnan(y[:, gone]).all() and torch.isfinite(y[:, ~gone]).all()


def codes(rng, *shape):
    return torch.from_numpy(rng.integers(-128, 128, shape).astype(np.int8))


def check(m, n, k, seed, bias=False):
    rng = np.random.default_rng(seed)
    xq, wq = codes(rng, m, k), codes(rng, n, k)
    sx = torch.from_numpy(rng.uniform(0.001, 0.1, m).astype(np.float32))
    sw = torch.from_numpy(rng.uniform(0.001, 0.1, n).astype(np.float32))
    b = bf16(rng, n) if bias else None
    y = B.nvfp4_int8_gemm(xq.to(DEV), sx.to(DEV), wq.to(DEV), sw.to(DEV), None if b is None else b.to(DEV))
    want, bound = D.int8_gemm(xq.numpy(), sx.numpy(), wq.numpy(), sw.numpy(), None if b is None else b.double().numpy())
    err = np.abs(y.cpu().double().numpy() - want)
    assert np.all(err <= bound), (np.argwhere(err > bound)[:4], err.max(), bound.min())


@pytest.mark.parametrize("m,n,k", [
    (1, 1, 16), (1, 17, 48), (2, 255, 112), (3, 1003, 528), (7, 300, 2080), (15, 513, 256), (16, 64, 1040), (17, 257, 128),
    (31, 100, 144), (32, 515, 640), (33, 1003, 528), (64, 33, 272), (65, 300, 1040), (100, 257, 96), (128, 511, 384),
    (333, 22003, 528), (700, 33000, 144), (2000, 9001, 656), (129, 400, 528), (255, 129, 1040), (257, 515, 656), (520, 770, 144), (1, 4099, 8208), (5, 20011, 128)])
@pytest.mark.parametrize("bias", [False, True])
def test_sizes(m, n, k, bias):
    check(m, n, k, seed=m * 100 + n + k, bias=bias)


@pytest.mark.parametrize("m", [1, 20, 200])
def test_extreme_sums_are_exact(m):
    """The largest K with every code at -128: 2^14 K just below 2^31, and one unit less in single places."""
    k = (1 << 17) - 16
    xq = torch.full((m, k), -128, dtype=torch.int8)
    wq = torch.full((3, k), -128, dtype=torch.int8)
    wq[1] = 127
    wq[2, ::2] = 127
    one = torch.ones(3)
    y = B.nvfp4_int8_gemm(xq.to(DEV), torch.ones(m, device=DEV), wq.to(DEV), one.to(DEV)).cpu()
    want = torch.from_numpy((xq[:1].numpy().astype(np.int64) @ wq.numpy().astype(np.int64).T).astype(np.float64))
    assert torch.equal(y, want.to(BF16).expand(m, 3))


def test_one_hot_rows_give_single_codes():
    n, k = 300, 256
    w = codes(np.random.default_rng(4), n, k)
    x = torch.eye(k, dtype=torch.int8)
    y = B.nvfp4_int8_gemm(x.to(DEV), torch.ones(k, device=DEV), w.to(DEV), torch.ones(n, device=DEV)).cpu()
    assert torch.equal(y, w.t().to(BF16))


@pytest.mark.parametrize("m", [1, 16, 40, 70, 150])
def test_output_is_written_exactly_and_alone(m):
    rng = np.random.default_rng(m)
    n, k = 45, 160
    buf = torch.full((m * n + 64,), 3.0, dtype=BF16, device=DEV)
    x, w = codes(rng, m, k).to(DEV), codes(rng, n, k).to(DEV)
    sx, sw = torch.full((m,), 0.01, device=DEV), torch.full((n,), 0.01, device=DEV)
    B.nvfp4_int8_gemm(x, sx, w, sw, out=buf[:m * n].view(m, n))
    assert torch.equal(buf[:m * n].view(m, n), B.nvfp4_int8_gemm(x, sx, w, sw)) and torch.all(buf[m * n:] == 3.0)


def test_empty_batch():
    e = lambda *s, dt=torch.int8: torch.empty(s, dtype=dt, device=DEV)
    assert B.nvfp4_int8_gemm(e(0, 32), e(0, dt=torch.float32), e(5, 32), e(5, dt=torch.float32)).shape == (0, 5)
    q, s = B.nvfp4_int8_quantize_rows(e(0, 32, dt=BF16))
    assert q.shape == (0, 32) and s.shape == (0,)


@pytest.mark.parametrize("m", [1, 33, 300])
def test_graph_replays(m):
    rng = np.random.default_rng(m)
    n, k = 1003, 528
    x, w = bf16(rng, m, k).to(DEV), codes(rng, n, k).to(DEV)
    sw = torch.full((n,), 0.01, device=DEV)
    held = []
    call = lambda: B.nvfp4_int8_gemm(*B.nvfp4_int8_quantize_rows(x), w, sw)
    graph = capture(lambda: held.append(call()))
    for _ in range(3):
        x.copy_(bf16(rng, m, k))
        graph.replay()
        torch.cuda.synchronize()
        got = held[-1].clone()
        assert torch.equal(got, call())


def test_given_stream_with_wide_input():
    rng = np.random.default_rng(9)
    x = bf16(rng, 20, 2 * 256).to(DEV)[:, ::2]           # the call makes its dense copy on the stream
    w, sw = codes(rng, 515, 256).to(DEV), torch.full((515,), 0.02, device=DEV)
    want = B.nvfp4_int8_gemm(*B.nvfp4_int8_quantize_rows(x), w, sw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q, s = B.nvfp4_int8_quantize_rows(x, stream=side)
    y = B.nvfp4_int8_gemm(q, s, w, sw, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_binding_refusals():
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8, device=DEV)
    f = lambda n: torch.zeros((n,), device=DEV)
    with pytest.raises(ValueError):
        B.nvfp4_int8_gemm(i8(4, 64), f(4), i8(8, 32), f(8))
    with pytest.raises(ValueError):
        B.nvfp4_int8_gemm(i8(4, 64), f(3), i8(8, 64), f(8))
    with pytest.raises(ValueError):
        B.nvfp4_int8_gemm(i8(4, 64), f(4), i8(8, 64), f(8), out=torch.zeros((8, 4), dtype=BF16, device=DEV))
    with pytest.raises(ValueError):
        B.nvfp4_int8_gemm(i8(4, 64), f(4), i8(8, 64).view(torch.uint8), f(8))
    with pytest.raises(B.NVFP4ShapeError):
        B.nvfp4_int8_gemm(i8(4, 72), f(4), i8(8, 72), f(8))
    with pytest.raises(B.NVFP4ShapeError):
        B.nvfp4_int8_quantize_rows(torch.zeros((4, 72), dtype=BF16, device=DEV))
