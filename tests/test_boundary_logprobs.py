"""Refusals of the log-probability calls, before any HIP call (no GPU needed),
and pins of their oracle."""

import numpy as np
import pytest
import torch

import oracle.logprobs_oracle as L
from nvfp4_w4a16_lm_amd import binding as B

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ALIAS, ERR_ARG = 0, 1, 2, 3, 4, 6
BASE = [0x10000000 * (i + 1) for i in range(16)]       # well-separated addresses, never touched


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def fwd(lib, **kw):
    a = dict(x=BASE[0], dt=0, M=4, V=1000, stride=1000, ids=BASE[1], temps=BASE[2], allowed=BASE[3], topk=5,
             ws=BASE[4], lp=BASE[5], rank=BASE[6], lse=BASE[7], ent=BASE[8], tlp=BASE[9], top=BASE[10])
    a.update(kw)
    return lib.nvfp4_logprobs(*a.values(), None)


def test_forward_refusals(lib):
    for name in ("x", "ws", "tlp", "top"):
        assert fwd(lib, **{name: 0}) == ERR_NULL, name
    assert fwd(lib, dt=3) == ERR_ARG and fwd(lib, dt=-1) == ERR_ARG
    for kw in (dict(M=-1), dict(M=(1 << 23) + 1), dict(V=0), dict(V=(1 << 30) + 1, stride=1 << 31),
               dict(stride=999), dict(topk=-1), dict(topk=65), dict(M=1 << 20, stride=1 << 21)):
        assert fwd(lib, **kw) == ERR_SHAPE, kw
    assert fwd(lib, x=BASE[0] + 1) == ERR_ALIGN
    assert fwd(lib, dt=2, x=BASE[0] + 2) == ERR_ALIGN
    for name in ("ids", "temps", "allowed", "lp", "rank", "lse", "ent", "tlp", "top"):
        assert fwd(lib, **{name: BASE[12] + 2}) == ERR_ALIGN, name
    assert fwd(lib, ws=BASE[4] + 8) == ERR_ALIGN
    for name in ("lp", "rank", "lse", "ent", "tlp", "top", "ws"):
        assert fwd(lib, **{name: BASE[0] + 7984}) == ERR_ALIAS, name      # the logits' last 16 bytes
    assert fwd(lib, lse=BASE[8]) == ERR_ALIAS
    assert fwd(lib, top=BASE[9] + 4) == ERR_ALIAS
    assert fwd(lib, lp=BASE[3] + 4 * 32 * 4 - 4) == ERR_ALIAS             # the mask's last word
    assert fwd(lib, M=0) == OK
    assert fwd(lib, M=0, x=0, ws=0, tlp=0, top=0) == OK
    assert lib.nvfp4_logprobs_workspace_bytes(1, 0, 0) == 0
    assert lib.nvfp4_logprobs_workspace_bytes(1, 100, 65) == 0
    assert lib.nvfp4_logprobs_workspace_bytes(1, 100, 5) >= 16


def bwd(lib, **kw):
    a = dict(x=BASE[0], dt=0, M=4, V=1000, stride=1000, ids=BASE[1], temps=BASE[2], allowed=BASE[3], lse=BASE[4],
             ent=BASE[5], dlp=BASE[6], dent=BASE[7], dlse=BASE[8], dx=BASE[9], dstride=1000)
    a.update(kw)
    return lib.nvfp4_logprobs_backward(*a.values(), None)


def test_backward_refusals(lib):
    for kw in (dict(x=0), dict(lse=0), dict(dx=0), dict(ent=0), dict(ids=0)):
        assert bwd(lib, **kw) == ERR_NULL, kw
    assert bwd(lib, dt=7) == ERR_ARG
    for kw in (dict(M=-1), dict(V=0), dict(stride=10), dict(dstride=999)):
        assert bwd(lib, **kw) == ERR_SHAPE, kw
    for name in ("temps", "allowed", "lse", "ent", "dlp", "dent", "dlse", "ids"):
        assert bwd(lib, **{name: BASE[12] + 1}) == ERR_ALIGN, name
    assert bwd(lib, dx=BASE[9] + 1) == ERR_ALIGN
    assert bwd(lib, dx=BASE[0] + 2) == ERR_ALIAS
    assert bwd(lib, dx=BASE[0], dstride=1001) == ERR_ALIAS                # in place needs the same stride
    assert bwd(lib, dx=BASE[4] - 64) == ERR_ALIAS
    assert bwd(lib, M=0, x=0, lse=0, dx=0) == OK


def test_binding_refusals():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):                                       # not a device tensor
        B.nvfp4_logprobs(x)
    with pytest.raises(TypeError):
        B.nvfp4_logprobs(x.double())
    with pytest.raises(B.NVFP4ShapeError):
        B.logprobs_buffers(2, 8, 65, "cpu")


def test_oracle_against_hand_values():
    x = np.log(np.float64([[1, 2, 5], [4, 4, 2]]))
    lp, rank, lse, ent, tlp, top = L.forward(x, [1, 0], 3)
    assert np.allclose(np.exp(lp), [0.25, 0.4]) and rank.tolist() == [2, 1]
    assert np.allclose(lse, np.log([8, 10]))
    assert np.allclose(ent, [0.125 * np.log(8) + 0.25 * np.log(4) - 0.625 * np.log(0.625),
                             0.8 * np.log(2.5) + 0.2 * np.log(5)])
    assert top.tolist() == [[2, 1, 0], [0, 1, 2]]
    allowed = L.allowed_bits(np.uint32([[0b101], [0b000]]), 3)
    lp, rank, lse, ent, tlp, top = L.forward(x, [1, 1], 2, allowed=allowed)
    assert lp.tolist() == [-np.inf, -np.inf] and rank.tolist() == [3, 1]
    assert np.allclose(lse[0], np.log(6)) and lse[1] == -np.inf and ent[1] == 0.0
    assert top.tolist() == [[2, 0], [-1, -1]] and np.all(tlp[1] == -np.inf)


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 7))
    ids, t = [3, 6], np.float64([0.8, 1.3])
    a, h, s = rng.standard_normal((3, 2))

    def loss(x):
        lp, _, lse, ent, _, _ = L.forward(x, ids, 0, t)
        return a * lp + h * ent + s * lse
    _, _, lse, ent, _, _ = L.forward(x, ids, 0, t)
    g, mag = L.backward(x, ids, lse, ent, a, h, s, t)
    for j in range(7):
        d = np.zeros_like(x)
        d[:, j] = 1e-5
        assert np.allclose((loss(x + d) - loss(x - d)) / 2e-5, g[:, j], atol=1e-8)
    assert np.all(mag >= np.abs(g) - 1e-12)


def test_workspace_of_every_accepted_size(lib):
    """0 means a refusal, also through logprobs_buffers: an empty batch is none, whatever the vocabulary."""
    for m in (0, 1, 2, 300, 1 << 23):
        for v in (1, 3000, 4096, 4097, 128256, 1 << 30):
            for topk in (0, 1, 64):
                assert lib.nvfp4_logprobs_workspace_bytes(m, v, topk) >= 16, (m, v, topk)
    b = B.logprobs_buffers(0, 128256, 5, "cpu")
    assert b.lse.shape == (0,) and b.top_ids.shape == (0, 5)
