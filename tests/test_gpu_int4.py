"""GPU parity of nvfp4_int4_gemm with the float64 oracle: group sizes, zero
points, both scale types, odd row and activation counts, K that ends inside a
chunk, bias, long K, and graph replays."""

import numpy as np
import pytest
import torch

import oracle.int4_oracle as Q
from nvfp4_w4a16_lm_amd import binding as B

from gpu_util import DEV
from test_gpu_graphs import capture

pytestmark = pytest.mark.gpu


def make(m, n, k, group, zeros, seed, scale_dtype=torch.bfloat16, bias=False):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (n, k))
    packed = Q.pack(codes, 1)
    g = k // group
    scales = torch.from_numpy(rng.uniform(0.001, 0.01, (n, g)) * rng.choice([-1, 1], (n, g))).to(scale_dtype)
    zp = Q.pack(rng.integers(0, 16, ((n + 7) // 8 * 8, g)), 0) if zeros else None
    x = torch.from_numpy(rng.standard_normal((m, k))).to(torch.bfloat16)
    b = torch.from_numpy(0.5 * rng.standard_normal(n)).to(torch.bfloat16) if bias else None
    return x, packed, scales, zp, b


def run(x, packed, scales, zp, b, out=None):
    dev = lambda a: None if a is None else (a if torch.is_tensor(a) else torch.from_numpy(a)).to(DEV)
    y = B.nvfp4_int4_gemm(dev(x), dev(packed), dev(scales), dev(zp), dev(b), out=out)
    torch.cuda.synchronize()
    return y


def check(m, n, k, group, zeros, seed, scale_dtype=torch.bfloat16, bias=False):
    x, packed, scales, zp, b = make(m, n, k, group, zeros, seed, scale_dtype, bias)
    y = run(x, packed, scales, zp, b)
    f64 = lambda t: None if t is None else t.to(torch.float64).numpy()
    want, bound = Q.gemm(f64(x), packed, f64(scales), zp, f64(b))
    err = np.abs(y.cpu().to(torch.float64).numpy() - want)
    assert np.all(err <= bound), (np.argwhere(err > bound)[:4], err.max(), bound.min())


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k,group", [
    (1, 1, 32, 32), (1, 7, 64, 64), (2, 33, 96, 32), (1, 100, 128, 128), (3, 65, 160, 32), (5, 31, 192, 64),
    (1, 515, 2080, 32), (16, 129, 640, 128), (17, 40, 512, 64), (33, 300, 1056, 32), (64, 100, 768, 256),
    (65, 50, 256, 128), (130, 17, 384, 64), (4, 96, 1024, 1024), (9, 70, 2080, 2080), (16, 1000, 4096, 128),
    (1, 32, 8192, 128), (48, 333, 1344, 64)])
def test_sizes(m, n, k, group, zeros):
    check(m, n, k, group, zeros, seed=m * 1000 + n + k, bias=(n % 2 == 1))


@pytest.mark.parametrize("group", [32, 64, 128, 512])
def test_f16_scales(group):
    check(7, 77, 1024, group, True, seed=group, scale_dtype=torch.float16, bias=True)


def test_every_code_and_zero_point_exactly():
    """x = one-hot rows: the output is one dequantized weight, exact before its bf16 rounding."""
    k, n, group = 128, 16, 32
    codes = (np.arange(n)[:, None] + np.arange(k)[None, :]) % 16
    zp = (3 * np.arange(n)[:, None] + np.arange(k // group)[None, :]) % 16
    scales = torch.full((n, k // group), 0.5, dtype=torch.bfloat16)
    for k0 in range(0, k, 64):
        x = torch.zeros((64, k), dtype=torch.bfloat16)
        x[torch.arange(64), k0 + torch.arange(64)] = 1.0
        y = run(x, Q.pack(codes, 1), scales, Q.pack(zp, 0), None).cpu().float().numpy()
        want = 0.5 * (codes - np.repeat(zp, group, 1))[:, k0:k0 + 64].T
        assert np.array_equal(y, want)


def test_many_rows_and_columns():
    check(16, 20011, 512, 128, False, seed=3)
    check(2, 70000, 256, 64, True, seed=4)


def test_infinite_activation_reaches_its_row_only():
    x, packed, scales, zp, _ = make(5, 64, 256, 64, True, 8)
    x[2, 17] = float("inf")
    y = run(x, packed, scales, zp, None).float().cpu()
    assert not torch.isfinite(y[2]).any() and torch.isfinite(y[[0, 1, 3, 4]]).all()


def test_output_buffer_is_written_exactly():
    m, n, k = 3, 45, 256
    x, packed, scales, zp, _ = make(m, n, k, 64, False, 9)
    buf = torch.full((m * n + 64,), 3.0, dtype=torch.bfloat16, device=DEV)
    out = buf[:m * n].view(m, n)
    run(x, packed, scales, zp, None, out=out)
    assert torch.equal(out, run(x, packed, scales, zp, None)) and torch.all(buf[m * n:] == 3.0)


def test_empty_batch():
    x, packed, scales, zp, _ = make(1, 16, 64, 32, False, 1)
    assert run(x[:0], packed, scales, zp, None).shape == (0, 16)


def test_graph_replays():
    m, n, k = 4, 1003, 1024
    x, packed, scales, zp, b = (None if t is None else (t if torch.is_tensor(t) else torch.from_numpy(t)).to(DEV)
                                for t in make(m, n, k, 128, True, 5, bias=True))
    y = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    graph = capture(lambda: B.nvfp4_int4_gemm(x, packed, scales, zp, b, out=y))
    for seed in (1, 2, 3):
        x.copy_(torch.randn((m, k), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, B.nvfp4_int4_gemm(x, packed, scales, zp, b))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(16, 700, 5120), (3, 5000, 8192), (20, 300, 5120), (40, 600, 4352), (64, 4500, 2336),
                                   (1, 100, 9216)])
def test_long_rows_in_phases(m, n, k, group):
    """K split over more wavefronts, chunks and phases than one pass holds (2336 = 9 x 256 + 32)."""
    if k % group:
        group = 32
    check(m, n, k, group, group != 128, seed=m + n + k + group)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k,group", [(1, 1, 1536, 32), (1, 70, 2048, 64), (2, 133, 1600, 32), (1, 515, 4096, 128),
                                         (2, 1001, 4096, 1024), (1, 99, 6144, 128), (1, 37, 8192, 8192),
                                         (1, 30011, 2048, 128), (2, 2000, 1984, 64),
                                         (1, 333, 1856, 32), (1, 10, 3776, 64), (2, 31, 2048, 2048)])
def test_one_and_two_rows(m, n, k, group, zeros):
    """The dot kernel: rows that fill a lane's one to four segments, wholly or partly."""
    check(m, n, k, group, zeros, seed=m + n + k + group, bias=(n % 2 == 1))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k,group", [
    (17, 13313, 96, 32), (33, 14001, 160, 32), (64, 13500, 320, 64), (48, 15007, 2080, 32), (30, 14111, 1152, 384),
    (40, 13333, 544, 544), (65, 8200, 256, 128), (200, 3511, 768, 256), (50, 14000, 1024, 128), (128, 7000, 32, 32),
    # more workgroups than compute units: two tiles per wavefront
    (64, 33000, 512, 128), (20, 33011, 352, 32), (256, 16500, 320, 64), (48, 66001, 128, 128), (18, 40007, 544, 32)])
def test_many_rows_of_both(m, n, k, group, zeros):
    """The tile kernel: odd and even counts of 256-k steps, K that ends inside one, rows that end inside a tile."""
    check(m, n, k, group, zeros, seed=m + n + k + group, bias=(n % 2 == 1))


def test_many_rows_of_both_f16_scales():
    check(33, 13999, 512, 64, True, seed=6, scale_dtype=torch.float16, bias=True)
    check(64, 34000, 384, 128, True, seed=7, scale_dtype=torch.float16)


@pytest.mark.parametrize("m,n,k,group", [(1, 64, 1888, 32), (1, 64, 3872, 32), (2, 64, 1888, 32), (4, 64, 160, 32),
                                         (3, 64, 192, 64), (5, 40, 384, 128), (40, 64, 160, 32), (20, 14000, 160, 32),
                                         (50, 13500, 384, 128), (64, 33000, 96, 96)])
def test_infinite_scale_of_the_last_group(m, n, k, group):
    """A step reaches past K there: what lies beyond is 0, not 0 times the scale."""
    x, packed, scales, zp, _ = make(m, n, k, group, True, m + k)
    scales[13, -1] = float("inf")
    y = run(x, packed, scales, zp, None).float().cpu()
    assert torch.isinf(y[:, 13]).all()
    y[:, 13] = 0
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k,group", [(2, 13201, 2336, 32), (3, 13313, 96, 32), (16, 14001, 160, 32), (9, 13500, 320, 64),
                                         (5, 16384, 1152, 384), (4, 20011, 544, 544), (16, 40001, 288, 32),
                                         (8, 99999, 128, 128), (8, 66000, 256, 128)])
def test_few_rows_on_many(m, n, k, group, zeros):
    """Up to 16 activation rows: the tile kernel, and the streamed one where its rounds would be uneven (66000)."""
    check(m, n, k, group, zeros, seed=m + n + k + group, bias=(n % 2 == 1))


@pytest.mark.parametrize("m,n,k,group", [(1, 1003, 1024, 128), (40, 13999, 544, 32), (16, 16000, 1024, 64), (64, 33000, 256, 128)])
def test_graph_replays_of_each_kernel(m, n, k, group):
    x, packed, scales, zp, b = (None if t is None else (t if torch.is_tensor(t) else torch.from_numpy(t)).to(DEV)
                                for t in make(m, n, k, group, True, 15, bias=True))
    y = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    graph = capture(lambda: B.nvfp4_int4_gemm(x, packed, scales, zp, b, out=y))
    for seed in (1, 2, 3):
        x.copy_(torch.randn((m, k), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, B.nvfp4_int4_gemm(x, packed, scales, zp, b))


def test_another_stream():
    x, packed, scales, zp, b = make(40, 14000, 512, 32, True, 16, bias=True)
    want = run(x, packed, scales, zp, b)
    dev = [(t if torch.is_tensor(t) else torch.from_numpy(t)).to(DEV) for t in (x, packed, scales, zp, b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = B.nvfp4_int4_gemm(*dev)
    side.synchronize()
    assert torch.equal(got, want)


KERNELS = [(1, 40, 512), (1, 30, 4096), (2, 33, 1024), (3, 50, 512), (9, 40, 4352), (16, 700, 5120), (20, 70, 1056),
           (40, 600, 1344), (64, 100, 768), (16, 14001, 320), (33, 14001, 160), (64, 33000, 512)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128, None])
@pytest.mark.parametrize("m,n,k", KERNELS)
def test_large_activation_on_a_zero_weight(m, n, k, group, zeros):
    """An activation of 2^18 in each group whose code is the zero point, among small whole numbers: every
    partial sum with an offset of 16 is a whole number below 2^24, so the result is exact before its
    one rounding to bf16, and the large activation leaves nothing."""
    group = k if group is None or k % group else group
    rng = np.random.default_rng(n + k)
    g = k // group
    codes, zp = rng.integers(0, 16, (n, k)), rng.integers(0, 16, (n, g)) if zeros else np.full((n, g), 8)
    x = rng.integers(-1, 2, (m, k)).astype(np.float64)
    at = group * np.arange(g) + rng.integers(0, group, g)
    if group == k:
        at = at[:1]
    codes[:, at] = zp
    x[:, at] = 2.0 ** 18 * rng.choice([-1, 1], (m, len(at)))
    scale = 2.0 ** rng.integers(-8, -6, (n, g))
    packed = Q.pack(codes, 1)
    pad = np.zeros(((n + 7) // 8 * 8, g), np.int64)
    pad[:n] = zp
    y = run(torch.from_numpy(x).to(torch.bfloat16), packed, torch.from_numpy(scale).to(torch.bfloat16),
            Q.pack(pad, 0) if zeros else None, None)
    want = x @ ((codes - np.repeat(zp, group, 1)) * np.repeat(scale, group, 1)).T
    # the groups' sums, scaled by powers of two, add exactly too
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(torch.bfloat16))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", KERNELS)
def test_activations_of_large_magnitude(m, n, k, group):
    """x = one-hot rows of 2^122: each output is one dequantized weight times it, finite."""
    if k % group:
        group = 32
    rng = np.random.default_rng(m + n)
    g = k // group
    codes, zp = rng.integers(0, 16, (n, k)), rng.integers(0, 16, ((n + 7) // 8 * 8, g))
    pos = rng.integers(0, k, m)
    x = torch.zeros((m, k), dtype=torch.bfloat16)
    x[torch.arange(m), torch.from_numpy(pos)] = 2.0 ** 122
    scale = torch.full((n, g), 2.0 ** -10, dtype=torch.bfloat16)
    y = run(x, Q.pack(codes, 1), scale, Q.pack(zp, 0), None).cpu().double().numpy()
    want = 2.0 ** 112 * (codes - np.repeat(zp[:n], group, 1))[:, pos].T
    assert np.array_equal(y, want)


@pytest.mark.parametrize("m,n,k,group", [(3, 66001, 4096, 128), (16, 70000, 4352, 256), (8, 80003, 5120, 5120),
                                         (5, 66000, 3840, 128), (9, 70001, 5248, 128)])
def test_few_rows_in_uneven_rounds(m, n, k, group):
    """Up to 16 rows where the tile kernel's last round would be mostly empty: streamed for K of 16 to 20
    chunks, tiles beside it.  (64 different rows, so that the host has little to make.)"""
    x, packed, scales, _, _ = make(m, 64, k, group, False, m + n)
    rows = np.arange(n) * 7 % 64
    want, bound = Q.gemm(x.to(torch.float64).numpy(), packed, scales.to(torch.float64).numpy())
    y = run(x, packed[rows], scales[torch.from_numpy(rows)], None, None).cpu().to(torch.float64).numpy()
    err = np.abs(y - want[:, rows])
    assert np.all(err <= bound[:, rows]), err.max()
