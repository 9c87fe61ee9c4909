"""Refusals of nvfp4_int4_gemm before any HIP call (no GPU needed), and pins of
its oracle."""

import numpy as np
import pytest
import torch

import oracle.int4_oracle as Q
from nvfp4_w4a16_lm_amd import binding as B

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ALIAS, ERR_ARG = 0, 1, 2, 3, 4, 6
X, P, S, Z, BIAS, Y = (0x10000000 * (i + 1) for i in range(6))


def call(**kw):
    a = dict(x=X, M=4, K=512, p=P, s=S, dt=0, z=Z, group=128, N=1000, b=BIAS, y=Y)
    a.update(kw)
    return B.load_library().nvfp4_int4_gemm(*a.values(), None)


def test_refusals():
    for name in ("x", "p", "s", "y"):
        assert call(**{name: 0}) == ERR_NULL, name
    assert call(dt=2) == ERR_ARG and call(dt=-1) == ERR_ARG
    for kw in (dict(M=-1), dict(K=16), dict(K=48, group=48), dict(K=0), dict(N=0), dict(group=0), dict(group=16),
               dict(group=96, K=960), dict(group=384), dict(group=-128), dict(N=1 << 31), dict(K=1 << 31)):
        assert call(**kw) == ERR_SHAPE, kw
    assert call(x=X + 8) == ERR_ALIGN
    assert call(p=P + 4) == ERR_ALIGN
    assert call(s=S + 1) == ERR_ALIGN
    assert call(z=Z + 2) == ERR_ALIGN
    assert call(b=BIAS + 1) == ERR_ALIGN
    assert call(y=Y + 2) == ERR_ALIGN
    assert call(y=X + 4 * 512 * 2 - 16) == ERR_ALIAS
    assert call(y=P + 1000 * 256 - 16) == ERR_ALIAS
    assert call(y=S - 4 * 1000 * 2 + 16) == ERR_ALIAS
    assert call(y=Z + 125 * 16 - 16) == ERR_ALIAS
    assert call(y=BIAS) == ERR_ALIAS
    assert call(M=0) == OK
    assert call(M=0, x=0, y=0) == OK
    assert call(M=0, group=512, z=0, b=0) == OK        # one scale per row


def test_binding_refusals():
    x = torch.zeros((1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):                     # not a device tensor
        B.nvfp4_int4_gemm(x, torch.zeros((4, 8), dtype=torch.int32), torch.zeros((4, 2), dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        B.nvfp4_int4_gemm(x.float(), torch.zeros((4, 8), dtype=torch.int32), torch.zeros((4, 2), dtype=torch.bfloat16))


def test_oracle_by_hand():
    codes = np.array([[0, 15, 8, 7, 1, 2, 3, 4]] * 4 + [[9] * 8] * 12).reshape(16, 8)
    words = Q.pack(codes, 1)
    assert words[0, 0] == np.int32(np.uint32(0x432178F0).view(np.int32))
    assert np.array_equal(Q.unpack(words, 1), codes)
    w, _ = Q.weight(words, np.array([[0.5]] * 16), None, 16)
    assert w[0].tolist() == [-4.0, 3.5, 0.0, -0.5, -3.5, -3.0, -2.5, -2.0]
    zeros = Q.pack(np.arange(16).reshape(16, 1), 0)
    assert np.array_equal(Q.unpack(zeros, 0)[:, 0], np.arange(16))
    w, z = Q.weight(words, np.array([[2.0]] * 16), zeros, 16)
    assert w[3].tolist() == [-6.0, 24.0, 10.0, 8.0, -4.0, -2.0, 0.0, 2.0] and z[9, 0] == 9
    y, bound = Q.gemm(np.ones((1, 8)), words, np.array([[2.0]] * 16), zeros)
    assert y[0, 3] == 32.0 and bound[0, 3] < 0.2
