"""GPU parity of nvfp4_logprobs and nvfp4_logprobs_backward with the float64
oracle: types, odd sizes, row strides and alignments, masks, rows that have
nothing, ties, given tokens outside the row, and the gradient against the
formula and against differences.  Whole numbers must be equal; the others lie
within bounds derived from float32's and the output type's rounding."""

import numpy as np
import pytest
import torch

import oracle.logprobs_oracle as L
from nvfp4_w4a16_lm_amd import binding as B

from gpu_util import DEV
from test_gpu_graphs import capture

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def make_logits(m, v, dtype, seed, pad=0, offset=0):
    """[m, v] view with row stride v + pad, starting `offset` elements into its storage."""
    g = torch.Generator().manual_seed(seed)
    flat = (3.0 * torch.randn(offset + m * (v + pad), generator=g)).to(dtype)
    x = flat.to(DEV)[offset:].view(m, v + pad)[:, :v]
    return x


def host(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def words_of(bits: np.ndarray) -> np.ndarray:
    m, v = bits.shape
    pad = np.zeros((m, (v + 31) // 32 * 32), np.uint64)
    pad[:, :v] = bits
    w = (pad.reshape(m, -1, 32) << np.arange(32, dtype=np.uint64)).sum(2)
    return w.astype(np.uint32)


def dev_words(bits):
    return torch.from_numpy(words_of(bits).view(np.int32)).to(DEV)


def check_forward(x, ids, topk, temps=None, bits=None, out=None):
    tid = None if ids is None else torch.tensor(ids, dtype=torch.int32, device=DEV)
    td = None if temps is None else torch.tensor(temps, dtype=F32, device=DEV)
    r = B.nvfp4_logprobs(x, tid, topk=topk, temperatures=td, allowed=None if bits is None else dev_words(bits),
                         out=out)
    torch.cuda.synchronize()
    t64 = None if temps is None else np.float32(temps).astype(np.float64)
    lp, rank, lse, ent, tlp, top = L.forward(host(x), ids, topk, t64, bits)
    b_s, b_lse, b_h = L.forward_bounds(host(x), t64, bits)
    got = [host(t) for t in r[:6]]
    assert np.array_equal(got[5].astype(np.int64), top), "alternatives"
    if ids is not None:
        assert np.array_equal(got[1].astype(np.int64), rank), "ranks"

    def close(g, want, bound, what):
        same = (g == want) | (np.isnan(g) & np.isnan(want))
        with np.errstate(invalid="ignore"):
            ok = same | (np.abs(g - want) <= bound)
        assert np.all(ok), f"{what}: {g[~ok][:4]} != {want[~ok][:4]} (bound {np.broadcast_to(bound, g.shape)[~ok][:4]})"
    raw, z = L.scaled(host(x), t64, bits)
    with np.errstate(invalid="ignore"):
        top_z = np.max(np.where(np.isnan(z), -np.inf, z), axis=1)
        top_z = np.where(np.isfinite(top_z), top_z, 0.0)
    close(got[2], lse, b_lse, "lse")
    close(got[3], ent, b_h, "entropy")
    if ids is not None:
        zi = np.array([z[i, j] if 0 <= j < z.shape[1] else 0.0 for i, j in enumerate(ids)])
        close(got[0], lp, b_s + 6 * U * np.where(np.isfinite(zi), np.abs(zi - top_z), 0.0)
              + 4 * U * np.where(np.isfinite(lp), np.abs(lp), 0.0), "logprobs")
    zt = np.where(top >= 0, np.take_along_axis(z, np.maximum(top, 0), 1), 0.0)
    zt = np.where(np.isfinite(zt) & (top >= 0), np.abs(zt - top_z[:, None]), 0.0)
    close(got[4], tlp, b_s[:, None] + 6 * U * zt + 4 * U * np.where(np.isfinite(tlp), np.abs(tlp), 0.0),
          "top logprobs")
    return r


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("m,v,topk,pad,offset", [
    (1, 1, 1, 0, 0), (3, 2, 5, 0, 1), (2, 7, 7, 1, 3), (5, 31, 3, 0, 0), (4, 33, 64, 2, 1), (3, 255, 20, 0, 0),
    (2, 4095, 1, 0, 0), (2, 4096, 8, 8, 0), (2, 4097, 64, 0, 5), (1, 32003, 20, 0, 0), (7, 32003, 0, 5, 1),
    (1030, 1003, 2, 0, 0), (1, 128256, 5, 0, 0), (33, 20000, 33, 0, 0)])
def test_forward_sizes(dtype, m, v, topk, pad, offset):
    x = make_logits(m, v, dtype, 100 * m + v, pad, offset)
    rng = np.random.default_rng(v)
    ids = rng.integers(0, v, m).astype(np.int32)
    temps = rng.uniform(0.5, 1.5, m).astype(np.float32) if m % 2 else None
    check_forward(x, ids, topk, temps)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("m,v,topk", [(6, 37, 40), (6, 1000, 20), (6, 9001, 64), (6, 70001, 5)])
def test_forward_masks_hide_whatever_they_cover(dtype, m, v, topk):
    x = make_logits(m, v, dtype, v)
    rng = np.random.default_rng(v + 1)
    bits = rng.random((m, v)) < 0.3
    bits[0] = False                                      # nothing allowed
    bits[1] = False
    bits[1, v - 1] = True                                # one token
    bits[2] = True
    ids = rng.integers(0, v, m).astype(np.int32)
    bits[3, ids[3]] = False                              # the given token is not allowed
    bits[4, ids[4]] = True
    hidden = torch.from_numpy(~bits).to(DEV)
    for bad in (float("nan"), float("inf"), float("-inf"), torch.finfo(dtype).min):
        check_forward(torch.where(hidden, torch.tensor(bad, dtype=dtype, device=DEV), x), ids, topk,
                      np.full(m, 0.7, np.float32), bits)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("v", [5, 600, 5001, 40000])
def test_forward_special_rows(dtype, v):
    m = 11
    x = make_logits(m, v, dtype, v + 2).contiguous()
    lowest = torch.finfo(dtype).min
    x[0] = float("-inf")
    x[1] = float("-inf")
    x[1, v // 2] = 1.5                                   # one finite logit: entropy 0
    x[2] = 0.0                                           # all equal
    x[3] = 0.0
    x[3, ::2] = -0.0                                     # equal too
    x[4] = lowest                                        # all of the type's lowest value: uniform
    x[5, 1:] = lowest
    x[6, v - 1] = float("nan")
    x[7, 0] = float("inf")
    x[8] = torch.finfo(dtype).max                        # overflows once scaled to base 2 (bf16, f32)
    x[9] = torch.linspace(-5, 5, v).to(dtype)            # rising: every group brings new alternatives
    ids = np.full(m, v // 2, np.int32)
    ids[10] = -1
    for topk in (0, 1, 20, 64):
        r = check_forward(x, ids, topk)
    assert int(r.token_ranks[10]) == 0 and float(r.token_logprobs[10]) == 0.0
    for bad in (v, -100, 2 ** 31 - 1):
        r = check_forward(x, np.full(m, bad, np.int32), 3)
        assert not r.token_ranks.any() and not r.token_logprobs.any()
    check_forward(x, None, 2)


def test_forward_temperatures_and_optional_outputs():
    x = make_logits(5, 3001, BF16, 9)
    check_forward(x, np.arange(5, dtype=np.int32), 4, np.float32([0.0, -1.0, 0.05, 4.0, 1.0]))
    nan_t = torch.tensor([float("nan")] * 5, device=DEV)
    one = B.nvfp4_logprobs(x, None, topk=3)
    got = B.nvfp4_logprobs(x, None, topk=3, temperatures=nan_t)
    for a, b in zip(one[2:6], got[2:6]):
        assert torch.equal(a, b)


def test_forward_empty_batch():
    x = torch.empty((0, 100), dtype=BF16, device=DEV)
    r = B.nvfp4_logprobs(x, torch.empty((0,), dtype=torch.int32, device=DEV), topk=3)
    assert r.lse.shape == (0,) and r.top_ids.shape == (0, 3)


def test_forward_same_bits_every_time_and_on_a_side_stream():
    x = make_logits(3, 128256, BF16, 11)
    ids = torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV)
    first = B.nvfp4_logprobs(x, ids, topk=20)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = B.logprobs_buffers(3, 128256, 20, DEV)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(side):
            B.nvfp4_logprobs(x, ids, topk=20, out=out)
        side.synchronize()
        for a, b in zip(first[:6], out[:6]):
            assert torch.equal(a, b)


GRAD_TYPES = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}


def run_backward(x, ids, dlp, dent, dlse, temps, bits, out=None):
    dev = lambda a, t=F32: None if a is None else torch.tensor(a, dtype=t, device=DEV)
    words = None if bits is None else dev_words(bits)
    tid, td = dev(ids, torch.int32), dev(temps)
    f = B.nvfp4_logprobs(x, tid, temperatures=td, allowed=words)
    g = B.nvfp4_logprobs_backward(x, tid, f.lse, f.entropy, dev(dlp), dev(dent), dev(dlse), td, words, out=out)
    torch.cuda.synchronize()
    return g, host(f.lse), host(f.entropy)


def check_backward(x, ids, dlp=None, dent=None, dlse=None, temps=None, bits=None, out=None):
    want_x = host(x)
    g, lse, ent = run_backward(x, ids, dlp, dent, dlse, temps, bits, out)
    t64 = None if temps is None else np.float32(temps).astype(np.float64)
    f64 = lambda a: None if a is None else np.float32(a).astype(np.float64)
    want, mag = L.backward(want_x, ids, lse, ent, f64(dlp), f64(dent), f64(dlse), t64, bits)
    _, z = L.scaled(want_x, t64, bits)
    z = np.where(np.isfinite(z), np.abs(z), 0.0)
    lse_mag = np.where(np.isfinite(lse), np.abs(lse), 0.0)[:, None]
    # log p within 3 u of |z| and |lse|, p relative to it, a few more roundings of each term;
    # below float32's normal range a result may become 0
    bound = mag * (4 * U * (z + lse_mag) + 16 * U) + GRAD_TYPES[x.dtype] * np.abs(want) * (1 + 2.0 ** -7)
    tiny = {BF16: 2.0 ** -126, F16: 2.0 ** -25, F32: 2.0 ** -126}[x.dtype]
    got = host(g)
    ok = np.abs(got - want) <= bound + tiny * 1.01
    assert np.all(ok), (got[~ok][:4], want[~ok][:4], bound[~ok][:4])
    return g


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("m,v,pad,offset", [(1, 1, 0, 0), (3, 5, 2, 1), (2, 31, 0, 0), (4, 4096, 0, 0),
                                            (3, 4099, 1, 3), (5, 9001, 0, 1), (2, 32003, 5, 0), (70, 513, 0, 0)])
def test_backward_sizes(dtype, m, v, pad, offset):
    x = make_logits(m, v, dtype, m + v, pad, offset)
    rng = np.random.default_rng(m + v)
    ids = rng.integers(0, v, m).astype(np.int32)
    ids[m // 2] = -1 if m > 1 else ids[0]
    dlp, dent, dlse = (rng.standard_normal(m) for _ in range(3))
    temps = rng.uniform(0.5, 1.5, m).astype(np.float32)
    check_backward(x, ids, dlp, None, None)
    check_backward(x, ids, dlp, dent, dlse, temps)
    check_backward(x, None, None, dent, None, temps)
    bits = rng.random((m, v)) < 0.4
    bits[0] = False
    bits[m - 1, ids[m - 1] if ids[m - 1] >= 0 else 0] = True
    check_backward(x, ids, dlp, dent, dlse, temps, bits)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_backward_strided_output_and_in_place(dtype):
    m, v = 5, 3003
    x = make_logits(m, v, dtype, 77, pad=3, offset=1)
    rng = np.random.default_rng(4)
    ids, dlp, dent = rng.integers(0, v, m).astype(np.int32), rng.standard_normal(m), rng.standard_normal(m)
    plain = check_backward(x, ids, dlp, dent).clone()
    buf = torch.full((m, v + 6), 7.0, dtype=dtype, device=DEV)
    check_backward(x, ids, dlp, dent, out=buf[:, 2:v + 2])
    assert torch.equal(buf[:, 2:v + 2], plain)
    assert torch.all(buf[:, :2] == 7.0) and torch.all(buf[:, v + 2:] == 7.0), "wrote outside its rows"
    check_backward(x, ids, dlp, dent, out=x)             # the gradient replaces the logits
    assert torch.equal(x, plain)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_backward_special_rows(dtype):
    m, v = 6, 700
    x = make_logits(m, v, dtype, 5).contiguous()
    x[0] = float("-inf")
    x[1] = float("-inf")
    x[1, 3] = 2.0
    x[2, ::3] = float("-inf")
    x[3] = 1.0
    ids = np.int32([3, 3, 3, 4, v, -5])
    check_backward(x, ids, np.ones(m), np.full(m, 0.3), np.full(m, -0.2))
    x[4, 7] = float("nan")                               # reaches every gradient of its row, no other row
    g, _, _ = run_backward(x, ids, np.ones(m), np.full(m, 0.3), None, None, None)
    assert torch.isnan(g[4]).all() and not torch.isnan(g[[0, 1, 2, 3, 5]]).any()


def test_backward_against_differences():
    """Central differences of the float64 forward, h = 2^-10: its error is h^2 / 6 times the
    third derivative of each term (log softmax and entropy: below 4 (1 + H) in size) plus the
    rounding of the difference."""
    m, v, h = 3, 40, 2.0 ** -10
    x = make_logits(m, v, F32, 21)
    rng = np.random.default_rng(2)
    ids = rng.integers(0, v, m).astype(np.int32)
    dlp, dent, dlse = (rng.standard_normal(m).astype(np.float32).astype(np.float64) for _ in range(3))
    temps = np.float64([0.75, 1.0, 1.5])
    g, _, _ = run_backward(x, ids, dlp, dent, dlse, temps, None)

    def loss(xs):
        lp, _, lse, ent, _, _ = L.forward(xs, ids, 0, temps)
        return dlp * lp + dent * ent + dlse * lse
    x64 = host(x)
    num = np.empty((m, v))
    for j in range(v):
        up, dn = x64.copy(), x64.copy()
        up[:, j] += h
        dn[:, j] -= h
        num[:, j] = (loss(up) - loss(dn)) / (2 * h)
    weight = (np.abs(dlp) + np.abs(dent) * (1 + np.log(v)) + np.abs(dlse))[:, None] / temps[:, None] ** 3
    assert np.all(np.abs(host(g) - num) <= weight * (4 * h * h / 6 + 2.0 ** -20))


def test_logprobs_graph_replays():
    m, v, topk = 4, 20011, 8
    x = make_logits(m, v, BF16, 1).contiguous()
    ids = torch.zeros((m,), dtype=torch.int32, device=DEV)
    out = B.logprobs_buffers(m, v, topk, DEV)
    dlp = torch.ones((m,), device=DEV)
    dx = torch.empty((m, v), dtype=BF16, device=DEV)

    def step():
        B.nvfp4_logprobs(x, ids, topk=topk, out=out)
        B.nvfp4_logprobs_backward(x, ids, out.lse, out.entropy, dlp, dentropy=dlp, out=dx)
    graph = capture(step)
    for seed in (2, 3, 4):
        x.copy_(make_logits(m, v, BF16, seed))
        ids.fill_(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out[:6]] + [dx.clone()]
        eager = B.nvfp4_logprobs(x, ids, topk=topk)
        edx = B.nvfp4_logprobs_backward(x, ids, eager.lse, eager.entropy, dlp, dentropy=dlp)
        torch.cuda.synchronize()
        for a, b in zip(got, [*eager[:6], edx]):
            assert torch.equal(a, b), f"replay {seed}"


@pytest.mark.parametrize("v", [4097, 128256])
def test_forward_empty_batch_of_a_long_vocabulary(v):
    """V beyond one segment of a row, where an empty batch's workspace has no segments."""
    x = torch.empty((0, v), dtype=BF16, device=DEV)
    r = B.nvfp4_logprobs(x, torch.empty((0,), dtype=torch.int32, device=DEV), topk=3)
    assert r.lse.shape == (0,) and r.top_ids.shape == (0, 3)
    g = B.nvfp4_logprobs_backward(x, torch.empty((0,), dtype=torch.int32, device=DEV), r.lse, r.entropy)
    assert g.shape == (0, v)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [9, 1000, 5001, 40000])
@pytest.mark.parametrize("temp", [None, 4.0])         # at 0.5 the log probability of -2^126 is -2^128, no float32
def test_forward_sums_far_below_the_maximum(dtype, v, temp):
    """Logits of +-2^126, whose scaling to base 2 is exact: the distance of an empty lane's sums, or
    of many low logits', to a later maximum passes float32, and they count as zero."""
    top = 2.0 ** 126
    x = torch.full((4, v), -top, dtype=dtype, device=DEV)
    x[0] = top                                           # uniform
    x[1, v - 1] = 0.0                                    # all the others at -top
    x[2, :v // 2] = 1.0
    x[3, 0] = top
    temps = None if temp is None else np.full(4, temp, np.float32)
    for topk in (0, 5):
        check_forward(x, np.int32([0, v - 1, 0, v - 1]), topk, temps)
        check_forward(x, np.int32([1, 0, v - 1, 0]), topk, temps)


LARGE = [3e9, 1e10, 1e15, 1e20, 1e30, 1e37, 5e37, 1.5e38]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [9, 1000, 5001, 40000])
@pytest.mark.parametrize("top", LARGE)
def test_forward_logits_of_large_magnitude(dtype, v, top):
    """Finite maxima and finite mask or padding values of any size, lanes full of them among the rows:
    a sum is relative to its own maximum exactly, not to the rounded product of it and log2(e) / T."""
    rng = np.random.default_rng(v)
    x = make_logits(7, v, dtype, v + 5).contiguous()
    x[0] = top                                           # uniform
    x[1, :v - 1] = -top                                  # one ordinary logit
    x[2, v // 2:] = -top
    x[3] = -top
    x[4, 0] = top
    x[4, 1:] = -top
    x[5][torch.from_numpy(rng.random(v) < 0.9).to(DEV)] = -top
    x[6] = x[6] * (top / 16)
    x[6, v // 3] = top
    ids = rng.integers(0, v, 7).astype(np.int32)
    for topk in (0, 5):
        check_forward(x, ids, topk)
        check_forward(x, ids, topk, np.float32([1.4, 0.8, 0.7, 2.0, 1.1, 0.9, 1.3]))
    check_forward(x, ids, 3, np.float32([1.4, 0.8, 0.7, 2.0, 1.1, 0.9, 1.3]), rng.random((7, v)) < 0.5)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("v", [9, 5001, 40000])
@pytest.mark.parametrize("temp", [1e-5, 1e-8, 1e-10, 1e-20, 1e-36])
def test_forward_low_temperatures(dtype, v, temp):
    """Greedy but for the name: z = logits / T passes 2^30 and every logit stays apart from the largest."""
    x = make_logits(4, v, dtype, v + 6)
    x[1] = torch.round(x[1])                             # many equal maxima
    x[2] = -x[2].abs() - 1.0
    ids = x.argmax(1).to(torch.int32).cpu().numpy()
    ids[3] = (ids[3] + 1) % v
    check_forward(x, ids, 4, np.full(4, temp, np.float32))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("v", [5, 1000, 4096, 5001, 40000])
def test_forward_infinite_temperature(dtype, v):
    """z = 0 for every finite logit, whether or not the row fills its last step: lse = log(count); what
    is not allowed, or -inf, still counts for nothing."""
    rng = np.random.default_rng(v)
    m = 5
    x = make_logits(m, v, dtype, v + 7).contiguous()
    x[1, ::2] = float("-inf")
    x[2] = float("-inf")
    x[3, v // 2:] = torch.finfo(dtype).min
    bits = rng.random((m, v)) < 0.5
    bits[4] = False
    temps = np.float32([np.inf, np.inf, np.inf, np.inf, 1.0])
    ids = rng.integers(0, v, m).astype(np.int32)
    for b in (None, bits):
        r = check_forward(x, ids, 5, temps, b)
        count = ((x > float("-inf")) & (True if b is None else torch.from_numpy(b).to(DEV)))[:2].sum(1)
        assert torch.allclose(r.lse[:2].double(), count.double().log(), rtol=1e-6, atol=1e-6)
        g = check_backward(x[:4], ids[:4], np.ones(4), np.full(4, 0.5), np.full(4, 0.25), temps[:4],
                           None if b is None else b[:4])
        assert not g.any()                               # 1 / T of anything
    check_forward(x, ids, 5, np.full(m, 3e38, np.float32), bits)


def check_backward_relative(x, ids, temps, bits=None, out=None):
    """The gradient against softmax relative to the row's maximum, for rows whose lse is too large for
    z - lse in float32 (or, further out, in float64); rows below that (header) among them as in
    check_backward, with the lse that the forward rounded."""
    m, v = x.shape
    rng = np.random.default_rng(v)
    dlp, dent, dlse = (rng.standard_normal(m).astype(np.float32).astype(np.float64) for _ in range(3))
    x64 = host(x)
    g, lse, ent = run_backward(x, ids, dlp, dent, dlse, temps, bits, out)
    t = np.float32(temps).astype(np.float64)[:, None]
    raw = x64 if bits is None else np.where(bits, x64, -np.inf)
    live = raw > -np.inf
    z = np.where(live, (np.where(live, raw, 0.0) - raw.max(1, keepdims=True)) / t, -np.inf)
    s = np.exp(z).sum(1, keepdims=True)
    p = np.exp(z) / s
    logp = np.where(live, z, 0.0) - np.log(s)
    c = lambda a: a[:, None]
    want = p * (c(dlse - dlp) - c(dent) * (logp + c(ent)))
    mag = p * (c(np.abs(dlse) + np.abs(dlp)) + c(np.abs(dent)) * (np.abs(logp) + c(np.abs(ent))))
    rows = np.arange(m)
    given = live[rows, ids]
    want[rows, ids] += np.where(given, dlp, 0.0)
    mag[rows, ids] += np.where(given, np.abs(dlp), 0.0)
    want, mag = want / t, mag / t
    # differences, quotients and log S as in the forward bounds, then as in check_backward; 2^y of a hardware
    # power and its argument's rounding, 3 u of |log p|
    rel = (v / 256.0 + v / 1024.0 + 40.0) * U
    bound = mag * (rel + 8 * U * np.abs(logp) + 16 * U) + GRAD_TYPES[x.dtype] * np.abs(want) * (1 + 2.0 ** -7)
    tiny = {BF16: 2.0 ** -126, F16: 2.0 ** -25, F32: 2.0 ** -126}[x.dtype]
    small = np.abs(lse) < (8192 if x.dtype == BF16 else 1024)
    if small.any():
        t64 = np.float32(temps).astype(np.float64)
        with np.errstate(all="ignore"):                  # the other rows of it are not used
            w2, m2 = L.backward(x64, ids, np.where(small, lse, 0.0), ent, dlp, dent, dlse, t64, bits)
        _, z2 = L.scaled(x64, t64, bits)
        z2 = np.where(np.isfinite(z2), np.abs(z2), 0.0)
        b2 = m2 * (4 * U * (z2 + np.abs(np.where(small, lse, 0.0))[:, None]) + 16 * U) + GRAD_TYPES[x.dtype] * np.abs(w2) * (1 + 2.0 ** -7)
        want, bound = np.where(c(small), w2, want), np.where(c(small), b2, bound)
    got = host(g)
    ok = np.abs(got - want) <= bound + tiny * 1.01
    assert np.all(ok), (got[~ok][:4], want[~ok][:4], bound[~ok][:4])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("v", [1, 9, 5001, 20011, 40000])
@pytest.mark.parametrize("offset,temp", [(0.0, 1e-3), (0.0, 3e-5), (2000.0, 1.0), (-40000.0, 0.7), (0.0, 1e-8)])
def test_backward_of_rows_with_a_large_lse(dtype, v, offset, temp):
    m = 4
    if dtype == F16:
        temp = max(temp, 1e-3)                           # 1 / T, and with it the gradient, within float16
    x = make_logits(m, v, F32, v + 9, pad=3, offset=1)
    if offset:
        x = x * 8.0 if dtype == BF16 else x              # bf16 logits lie 8 and more apart there
        x = x + offset
        top = x.amax(1, keepdim=True)
        x = torch.where(x > top - 30, x, torch.full_like(x, float("-inf")))
    x = x.to(dtype)
    if offset == 0.0:                                    # near ties: gradients that are not all 0 or 1
        x[1] = torch.round(x[1])
        x[2] = x.amax(1)[2]
    ids = x.argmax(1).cpu().numpy().astype(np.int32)
    ids[3] = (ids[3] + 1) % v
    temps = np.float32([temp, temp, temp, temp])
    check_backward_relative(x, ids, temps)
    bits = np.random.default_rng(v).random((m, v)) < 0.5
    bits[np.arange(m), x.argmax(1).cpu().numpy()] = True
    check_backward_relative(x, ids, temps, bits)
    check_backward_relative(x, ids, temps, bits, out=x)  # in place: the row is read before it is written


def test_backward_mixes_rows_of_either_kind():
    """Rows summed again beside ordinary ones, and a row whose lse overflows."""
    m, v = 6, 30000
    x = make_logits(m, v, F32, 3)
    x[1] += 5000.0
    x[4] -= 1e6
    temps = np.float32([1.0, 1.0, 1e-3, 0.8, 1.0, 1e-38])
    check_backward_relative(x, np.arange(m, dtype=np.int32), temps)


def test_workspace_kept_for_the_largest_batch():
    """One workspace of the largest batch for every smaller one, and nothing behind it is written."""
    v, topk, most = 70001, 20, 2100
    size = int(B.load_library().nvfp4_logprobs_workspace_bytes(most, v, topk))
    ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    x = make_logits(most, v, BF16, 21)
    ids = torch.arange(most, dtype=torch.int32, device=DEV) % v
    for m in (most, 2048, 2047, 1025, 1024, 700, 64, 2, 1):
        want = B.nvfp4_logprobs(x[:m], ids[:m], topk=topk)
        got = B.nvfp4_logprobs(x[:m], ids[:m], topk=topk, out=B.logprobs_buffers(m, v, topk, DEV)._replace(workspace=ws[:size]))
        assert all(torch.equal(a, b) for a, b in zip(got[:6], want[:6])), m
        assert torch.all(ws[size:] == 0xA5)
