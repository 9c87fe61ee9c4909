"""Refusals of the int8, linear cross entropy and gated feed-forward calls before
any HIP call (no GPU needed), their workspace sizes, and pins of their oracle."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle.dense_oracle as D
from nvfp4_w4a16_lm_amd import binding as B

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ALIAS = 0, 1, 2, 3, 4
P = [0x1000000000 * (i + 1) for i in range(16)]          # far apart; no call gets past its checks


def lib():
    return B.load_library()


def quant(**kw):
    a = dict(a=P[0], R=4, K=512, q=P[1], s=P[2])
    a.update(kw)
    return lib().nvfp4_int8_quantize_rows(*a.values(), None)


def gemm(**kw):
    a = dict(xq=P[0], sx=P[1], M=4, K=512, wq=P[2], sw=P[3], N=1001, b=P[4], y=P[5])
    a.update(kw)
    return lib().nvfp4_int8_gemm(*a.values(), None)


def ce(**kw):
    a = dict(x=P[0], M=4, K=512, w=P[1], V=1001, b=P[2], t=P[3], ws=P[4], loss=P[5], lse=P[6], st=P[7])
    a.update(kw)
    return lib().nvfp4_linear_ce(*a.values(), None)


def ceb(**kw):
    a = dict(x=P[0], M=4, K=512, w=P[1], V=1001, b=P[2], t=P[3], st=P[4], dl=P[5], de=P[6], ws=P[7], dx=P[8], dw=P[9],
             db=P[10])
    a.update(kw)
    return lib().nvfp4_linear_ce_backward(*a.values(), None)


def ffn(**kw):
    a = dict(x=P[0], T=4, H=512, w13=P[1], w2=P[2], I=1024, h=P[3], act=P[6], ws=P[4], y=P[5])
    a.update(kw)
    return lib().nvfp4_gated_ffn(*a.values(), None)


def ffnb(**kw):
    a = dict(x=P[0], T=4, H=512, h=P[1], act=P[9], w13=P[2], w2=P[3], I=1024, dy=P[4], ws=P[5], dx=P[6], dw13=P[7],
             dw2=P[8])
    a.update(kw)
    return lib().nvfp4_gated_ffn_backward(*a.values(), None)


def test_int8_refusals():
    for n in ("a", "q", "s"):
        assert quant(**{n: 0}) == ERR_NULL
    for kw in (dict(R=-1), dict(K=0), dict(K=24), dict(K=1 << 17), dict(R=(1 << 23) + 1)):
        assert quant(**kw) == ERR_SHAPE, kw
    assert quant(a=P[0] + 8) == ERR_ALIGN and quant(q=P[1] + 8) == ERR_ALIGN and quant(s=P[2] + 2) == ERR_ALIGN
    assert quant(q=P[0] + 4 * 512 * 2 - 16) == ERR_ALIAS and quant(s=P[1] + 4 * 512 - 4) == ERR_ALIAS
    assert quant(R=0, a=0, q=0, s=0) == OK
    for n in ("xq", "sx", "wq", "sw", "y"):
        assert gemm(**{n: 0}) == ERR_NULL, n
    for kw in (dict(M=-1), dict(M=(1 << 22) + 1), dict(N=0), dict(K=8), dict(K=520), dict(K=1 << 17), dict(N=1 << 31),
               dict(M=1 << 22, N=1 << 16)):
        assert gemm(**kw) == ERR_SHAPE, kw
    for n in ("xq", "wq", "y"):
        assert gemm(**{n: P[7] + 8}) == ERR_ALIGN, n
    for n in ("sx", "sw"):
        assert gemm(**{n: P[7] + 2}) == ERR_ALIGN, n
    assert gemm(b=P[4] + 1) == ERR_ALIGN
    for at in (P[0] + 4 * 512 - 16, P[1], P[2] + 1001 * 512 - 16, P[3] + 1001 * 4 - 4, P[4]):
        assert gemm(y=at // 16 * 16) == ERR_ALIAS
    assert gemm(M=0) == OK and gemm(M=0, xq=0, sx=0, y=0) == OK


def test_linear_ce_refusals():
    for n in ("x", "w", "t", "ws", "loss", "st"):
        assert ce(**{n: 0}) == ERR_NULL, n
    for n in ("x", "w", "t", "st", "dl", "ws"):
        assert ceb(**{n: 0}) == ERR_NULL, n
    for kw in (dict(M=-1), dict(M=(1 << 22) + 1), dict(V=0), dict(V=(1 << 30) + 1), dict(K=8), dict(K=520),
               dict(K=(1 << 20) + 16), dict(V=1 << 30, K=144), dict(M=1 << 22, V=(1 << 15) + 1), dict(M=1 << 22, K=1 << 16)):
        assert ce(**kw) == ERR_SHAPE and ceb(**kw) == ERR_SHAPE, kw
    for n in ("x", "w", "ws"):
        assert ce(**{n: P[11] + 8}) == ERR_ALIGN and ceb(**{n: P[11] + 8}) == ERR_ALIGN, n
    assert ce(st=P[7] + 4) == ERR_ALIGN and ceb(st=P[4] + 4) == ERR_ALIGN
    assert ce(b=P[2] + 1) == ERR_ALIGN and ce(loss=P[5] + 2) == ERR_ALIGN and ce(lse=P[6] + 2) == ERR_ALIGN
    for n in ("dx", "dw"):
        assert ceb(**{n: P[11] + 8}) == ERR_ALIGN, n
    assert ceb(dl=P[5] + 2) == ERR_ALIGN and ceb(db=P[10] + 1) == ERR_ALIGN and ceb(de=P[6] + 2) == ERR_ALIGN
    assert ce(loss=P[6]) == ERR_ALIAS and ce(ws=P[1] + 1001 * 1024 - 16) == ERR_ALIAS and ce(st=P[3]) == ERR_ALIAS
    assert ceb(dx=P[0]) == ERR_ALIAS and ceb(dw=P[1]) == ERR_ALIAS and ceb(db=P[9] + 64) == ERR_ALIAS
    assert ceb(dx=P[7]) == ERR_ALIAS and ceb(dw=P[5]) == ERR_ALIAS
    assert ce(M=0) == OK and ce(M=0, x=0, t=0, ws=0, loss=0, lse=0, st=0) == OK and ceb(M=0) == OK
    assert ceb(dx=0, dw=0, db=0) == OK                   # nothing asked for
    size = lib().nvfp4_linear_ce_workspace_bytes
    assert size(4, 1001, 8, 0) == 0 and size(-1, 1001, 512, 0) == 0 and size(4, 1001, 512, 2) == 0
    assert size(0, 1001, 512, 1) >= 16
    for m, v, k in ((1, 1, 16), (17, 32003, 512), (4096, 128256, 4096), (4194304, 1000, 16), (1, 1 << 30, 16)):
        assert size(m, v, k, 1) >= size(m, v, k, 0) >= 2 * m * k


def test_gated_ffn_refusals():
    for n in ("x", "w13", "w2", "ws", "y", "h", "act"):  # h and act: both or neither
        assert ffn(**{n: 0}) == ERR_NULL, n
    for n in ("x", "h", "act", "w13", "w2", "dy", "ws"):
        assert ffnb(**{n: 0}) == ERR_NULL, n
    for kw in (dict(T=-1), dict(T=(1 << 22) + 1), dict(H=8), dict(H=520), dict(I=0), dict(I=24), dict(H=(1 << 20) + 16),
               dict(I=(1 << 19) + 16), dict(H=1 << 16, I=1 << 14), dict(T=1 << 22, H=1 << 16, I=16), dict(T=1 << 22, H=16, I=1 << 15)):
        assert ffn(**kw) == ERR_SHAPE and ffnb(**kw) == ERR_SHAPE, kw
    for n in ("x", "w13", "w2", "h", "act", "ws", "y"):
        assert ffn(**{n: P[11] + 8}) == ERR_ALIGN, n
    for n in ("x", "h", "act", "w13", "w2", "dy", "ws", "dx", "dw13", "dw2"):
        assert ffnb(**{n: P[11] + 8}) == ERR_ALIGN, n
    assert ffn(y=P[0]) == ERR_ALIAS and ffn(h=P[1] + 2 * 1024 * 512 * 2 - 16) == ERR_ALIAS
    assert ffn(ws=P[3] + 4 * 2048 * 4 - 16) == ERR_ALIAS and ffn(act=P[3] + 64) == ERR_ALIAS
    assert ffnb(dx=P[4]) == ERR_ALIAS and ffnb(dw2=P[7] + 1024) == ERR_ALIAS and ffnb(dw13=P[1]) == ERR_ALIAS
    assert ffn(T=0) == OK and ffn(T=0, x=0, h=0, act=0, ws=0, y=0) == OK and ffnb(T=0) == OK
    assert ffnb(dx=0, dw13=0, dw2=0) == OK
    size = lib().nvfp4_gated_ffn_workspace_bytes
    assert size(4, 512, 24, 0) == 0 and size(4, 512, 1024, -1) == 0 and size(0, 512, 1024, 0) >= 16
    assert size(333, 2080, 5616, 1) >= size(333, 2080, 5616, 0) >= 2 * 333 * 5616


@pytest.mark.parametrize("back", [0, 1])
@pytest.mark.parametrize("call,a,b", [
    ("linear_ce", 32003, 512), ("linear_ce", 32003, 2080), ("linear_ce", 128256, 4096), ("linear_ce", 151936, 16),
    ("linear_ce", 1, 16), ("linear_ce", 1 << 20, 64), ("gated_ffn", 4096, 14336), ("gated_ffn", 2080, 5616), ("gated_ffn", 64, 96),
    ("gated_ffn", 16, 16), ("gated_ffn", 512, 1024), ("gated_ffn", 16384, 16), ("gated_ffn", 16, 65536)])
def test_workspace_of_a_batch_serves_every_smaller_one(call, a, b, back):
    """Sizes do not fall as the batch grows, and the backward pass's is the larger one."""
    size = getattr(lib(), f"nvfp4_{call}_workspace_bytes")
    rng = np.random.default_rng(a + b)
    ms = sorted({*range(2200), *(2 ** rng.uniform(11, 17, 300)).astype(int).tolist(), *(1 << e for e in range(11, 18))})
    last = 0
    for m in ms:
        n = size(m, a, b, back)
        assert n >= last and n >= size(m, a, b, 0) >= 16, (m, n, last)
        last = n


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refusals():
    t = torch.zeros((4,), dtype=torch.int32)
    with pytest.raises(ValueError):                      # not device tensors
        B.nvfp4_int8_quantize_rows(bf(4, 64))
    with pytest.raises(ValueError):
        B.nvfp4_int8_gemm(torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4), torch.zeros((8, 64), dtype=torch.int8),
                          torch.zeros(8))
    with pytest.raises(ValueError):
        B.nvfp4_linear_ce(bf(4, 64), bf(100, 64), t)
    with pytest.raises(ValueError):
        B.nvfp4_gated_ffn(bf(4, 64), bf(64, 64), bf(64, 32))
    with pytest.raises(TypeError):
        B.nvfp4_linear_ce(bf(4, 64).float(), bf(100, 64), t)
    with pytest.raises(TypeError):
        B.nvfp4_gated_ffn(bf(4, 64).half(), bf(64, 64), bf(64, 32))
    with pytest.raises(B.NVFP4ShapeError):
        B.linear_ce_workspace(4, 100, 72, "cpu")
    with pytest.raises(B.NVFP4ShapeError):
        B.gated_ffn_workspace(4, 64, 40, "cpu")


# ---------------------------------------------------------------------------
# The oracle
# ---------------------------------------------------------------------------

def bf16(rng, *shape, sigma=1.0):
    return torch.from_numpy(sigma * rng.standard_normal(shape)).to(torch.bfloat16).double().numpy()


def test_int8_codes_by_hand():
    a = np.array([[127.0, 0.5, 1.5, -2.5, 63.5, -127.0, 0.25, 126.0], [0.0] * 8, [2.0, -1.0, 0.0, 1.0, 0.5, 0.25, -0.125, 2.0]])
    q, s = D.int8_quantize_rows(a)
    assert q[0].tolist() == [127, 0, 2, -2, 64, -127, 0, 126] and s[0] == 1.0
    assert q[1].tolist() == [0] * 8 and s[1] == np.float32(1e-12)
    assert q[2].tolist() == [127, -64, 0, 64, 32, 16, -8, 127]
    y, b = D.int8_gemm(q[:1], s[:1], q[2:], s[2:], np.array([1.0]))
    want = Fraction(int((q[0].astype(int) * q[2].astype(int)).sum())) * Fraction(float(s[0])) * Fraction(float(s[2])) + 1
    assert abs(Fraction(y[0, 0]) - want) < Fraction(1, 10 ** 12) and b[0, 0] < 2.0 ** -7 * abs(y[0, 0])


def test_int8_rows_that_are_not_finite():
    a = np.ones((3, 16))
    a[0, 3], a[2, 5] = np.nan, -np.inf
    q, s = D.int8_quantize_rows(a)
    assert np.isnan(s[[0, 2]]).all() and not q[[0, 2]].any() and np.all(q[1] == 127) and np.isfinite(s[1])
    y, _ = D.int8_gemm(q, s, q[1:2], s[1:2])
    assert np.isnan(y[[0, 2]]).all() and abs(y[1, 0] - 16) < 1e-5


def test_float32_codes_are_those_of_the_exact_ratio():
    """One float32 division against exact rational arithmetic, over every significand of the maximum and of the
    element, and the element's scales at which it has a nonzero code."""
    amax = np.arange(128, 256, dtype=np.float64)
    for j in range(0, 9):
        v = np.arange(128, 256, dtype=np.float64) * 2.0 ** -j
        got = np.rint((np.float32(127) * v.astype(np.float32))[None, :] / amax.astype(np.float32)[:, None])
        got = got.clip(-127, 127).astype(int)
        num = (2 * 127 * np.arange(128, 256, dtype=np.int64))[None, :]           # 2 * 127 v 2^j
        den = (amax.astype(np.int64) << j)[:, None]                              # amax 2^j: ratio = num / (2 den)
        floor = num // (2 * den)
        rem2 = num - 2 * den * floor                                             # twice the remainder, against den
        want = floor + ((rem2 > den) | ((rem2 == den) & (floor % 2 == 1)))
        assert np.array_equal(got, np.minimum(want, 127)), j


def test_linear_ce_against_torch_and_differences():
    rng = np.random.default_rng(1)
    x, w, bias = bf16(rng, 6, 16), bf16(rng, 11, 16, sigma=0.5), bf16(rng, 11)
    t = np.array([3, -1, 10, 0, 11, 5])
    dloss, dlse = rng.standard_normal(6), rng.standard_normal(6)
    loss, lse, bl, be = D.linear_ce(x, w, t, bias)
    tx, tw, tb = (torch.from_numpy(a).requires_grad_() for a in (x, w, bias))
    z = tx @ tw.T + tb
    keep = torch.from_numpy((t >= 0) & (t < 11))
    ref = torch.nn.functional.cross_entropy(z, torch.from_numpy(np.where(keep, t, 0)), reduction="none") * keep
    tl = torch.logsumexp(z, 1) * keep
    assert np.allclose(loss, ref.detach()) and np.allclose(lse, tl.detach())
    assert np.all(bl < 1e-4) and loss[1] == loss[4] == bl[1] == 0
    (ref @ torch.from_numpy(dloss) + tl @ torch.from_numpy(dlse)).backward()
    (dx, dw, db), bounds = D.linear_ce_backward(x, w, t, dloss, dlse, bias)
    for a, b in ((dx, tx), (dw, tw), (db, tb)):
        assert np.allclose(a, b.grad, atol=1e-12)
    f = lambda x_, w_, b_: (lambda r: r[0] @ dloss + r[1] @ dlse)(D.linear_ce(x_, w_, t, b_))
    for which, grad in ((0, dx), (1, dw), (2, db)):
        args = [x, w, bias]
        d = rng.standard_normal(args[which].shape)
        up, down = list(args), list(args)
        up[which], down[which] = args[which] + 1e-5 * d, args[which] - 1e-5 * d
        assert abs((f(*up) - f(*down)) / 2e-5 - (grad * d).sum()) < 1e-7


def test_linear_ce_with_masked_tokens():
    rng = np.random.default_rng(2)
    x, w = bf16(rng, 3, 16), bf16(rng, 5, 16)
    bias = np.array([0.0, -np.inf, 1.0, -np.inf, 0.5])
    loss, lse, _, _ = D.linear_ce(x, w, np.array([0, 1, 2]), bias)
    assert np.isfinite(loss[[0, 2]]).all() and loss[1] == np.inf and np.isfinite(lse).all()
    (dx, dw, db), _ = D.linear_ce_backward(x, w, np.array([0, 1, 2]), np.ones(3), None, bias)
    assert np.all(db[[1, 3]] == 0) and np.all(dw[[1, 3]] == 0) and np.isfinite(dx).all()


def shared_targets(m, v, k, seed):
    """Rows that share a few targets (in no order, so in all groups of rows), their dloss such that each target's dz add up
    to about nothing: its column of db is a small sum of large terms."""
    rng = np.random.default_rng(seed)
    x, w, bias = bf16(rng, m, k), bf16(rng, v, k, sigma=0.5 / np.sqrt(k)), bf16(rng, v, sigma=0.2)
    t = rng.choice(np.linspace(0, v - 1, max(1, min(7, m // 4))).astype(int), m)
    dloss = np.where(rng.random(m) < 0.5, 1.0, -1.0) * rng.uniform(0.5, 1.0, m)
    z = x @ w.T + bias
    p = np.exp(z[np.arange(m), t] - np.log(np.exp(z).sum(1)))
    for u in np.unique(t):
        rows = np.nonzero(t == u)[0]
        dloss[rows[-1]] = -(dloss[rows[:-1]] * (1 - p[rows[:-1]])).sum() / (1 - p[rows[-1]])
    return x, w, bias, t, dloss.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("m,v,k", [(5, 300, 16), (20, 1003, 64), (130, 1003, 16), (700, 2003, 144)])
def test_bound_of_the_bias_gradient_tells_rounded_targets(m, v, k):
    """db summed from dz as the products take it, with the targets' dz rounded, is outside its bound; with them
    unrounded it is inside."""
    x, w, bias, t, dloss = shared_targets(m, v, k, seed=m)
    (_, _, db), (_, _, bound) = D.linear_ce_backward(x, w, t, dloss, None, bias)
    z = x @ w.T + bias
    dz = np.exp(z - z.max(1, keepdims=True))
    dz *= (dloss / dz.sum(1))[:, None]
    one = np.zeros_like(dz)
    one[np.arange(m), t] = 1.0
    dz -= dloss[:, None] * one
    low = lambda a: torch.from_numpy(a).to(torch.bfloat16).double().numpy()
    off = lambda terms: np.abs(low(terms.sum(0)) - db) / bound
    assert off(np.where(one > 0, dz, low(dz))).max() <= 1.0
    lost = off(low(dz))
    assert lost[np.unique(t)].max() > 2.0 and np.delete(lost, np.unique(t)).max() <= 1.0


def tied_targets(m, v, k, seed):
    """Few targets, of larger weights than the other tokens.  Rows of a target share their x, and their dz at it add up to
    about nothing: its row of dw is a small sum of large terms."""
    x, w, bias, t, _ = shared_targets(m, v, k, seed)
    rng = np.random.default_rng(seed + 1)
    targets = np.unique(t)
    x = bf16(rng, v, k)[t]
    w[:] = bf16(rng, v, k, sigma=0.02)
    w[targets] = bf16(rng, len(targets), k, sigma=1.2 / np.sqrt(k))
    dloss = np.where(rng.random(m) < 0.5, 1.0, -1.0) * rng.uniform(0.5, 1.0, m)
    for u in targets:
        rows = np.nonzero(t == u)[0]
        z = x[rows[0]] @ w.T + bias
        p = np.exp(z[u] - np.log(np.exp(z).sum()))
        # one row alone: a dz nearly half a step (2^-8) above 161/128
        dloss[rows[-1]] = -dloss[rows[:-1]].sum() if len(rows) > 1 else -(161 / 128 + 0.95 / 256) / (1.0 - p)
    return x, w, bias, t, dloss.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("m,v,k", [(1, 1003, 64), (5, 300, 16), (20, 1003, 64), (130, 4003, 16), (700, 6003, 144)])
def test_bounds_of_the_gradients_tell_rounded_targets(m, v, k):
    """dx and dw from dz rounded everywhere are outside their bounds; with the targets' dz unrounded inside."""
    x, w, bias, t, dloss = tied_targets(m, v, k, seed=m)
    (dx, dw, _), (bx, bw, _) = D.linear_ce_backward(x, w, t, dloss, None, bias)
    z = x @ w.T + bias
    dz = np.exp(z - z.max(1, keepdims=True))
    dz *= (dloss / dz.sum(1))[:, None]
    one = np.zeros_like(dz)
    one[np.arange(m), t] = 1.0
    dz -= dloss[:, None] * one
    low = lambda a: torch.from_numpy(a).to(torch.bfloat16).double().numpy()
    off = lambda q: [(np.abs(low(y) - want) / bound).max() for y, want, bound in ((q @ w, dx, bx), (q.T @ x, dw, bw))]
    assert max(off(np.where(one > 0, dz, low(dz)))) <= 1.0
    lost = off(low(dz))
    assert min(lost) > 1.2, lost


def test_gated_ffn_against_torch_and_differences():
    rng = np.random.default_rng(3)
    x, w13, w2, dy = bf16(rng, 5, 16), bf16(rng, 64, 16), bf16(rng, 16, 32), bf16(rng, 5, 16)
    (y, h, a), _ = D.gated_ffn(x, w13, w2)
    tx, t13, t2 = (torch.from_numpy(a).requires_grad_() for a in (x, w13, w2))
    g, u = (tx @ t13.T).chunk(2, 1)
    ref = (torch.nn.functional.silu(g) * u) @ t2.T
    assert np.allclose(y, ref.detach()) and np.allclose(h, torch.cat((g, u), 1).detach())
    (ref * torch.from_numpy(dy)).sum().backward()
    grads, _ = D.gated_ffn_backward(x, h, a, w13, w2, dy)
    for a, b in zip(grads, (tx, t13, t2)):
        assert np.allclose(a, b.grad, atol=1e-12)
    f = lambda *a: (D.gated_ffn(*a)[0][0] * dy).sum()
    for which, grad in enumerate(grads):
        args = [x, w13, w2]
        d = rng.standard_normal(args[which].shape)
        up, down = list(args), list(args)
        up[which], down[which] = args[which] + 1e-6 * d, args[which] - 1e-6 * d
        assert abs((f(*up) - f(*down)) / 2e-6 - (grad * d).sum()) < 1e-5 * (1 + abs((grad * d).sum()))
