"""Refusals of nvfp4_moe_w4a16_decode before any HIP call (no GPU needed), and
pins of its routing oracle."""

import numpy as np
import pytest
import torch

import oracle.moe_decode_oracle as D
from nvfp4_w4a16_lm_amd import binding as B

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ALIAS, ERR_ARG = 0, 1, 2, 3, 4, 6
BASE = [0x10000000 * (i + 1) for i in range(16)]


def call(**kw):
    a = dict(x=BASE[0], T=4, H=512, r=BASE[1], rt=2, E=8, topk=2, scoring=0, renorm=1, bias=BASE[2], scale=1.0,
             p13=BASE[3], s13=BASE[4], g13=BASE[5], p2=BASE[6], s2=BASE[7], g2=BASE[8], I=256, ws=BASE[9],
             out=BASE[10], ids=BASE[11], w=BASE[12])
    a.update(kw)
    return B.load_library().nvfp4_moe_w4a16_decode(*a.values(), None)


def test_refusals():
    for name in ("x", "r", "p13", "s13", "g13", "p2", "s2", "g2", "ws", "out"):
        assert call(**{name: 0}) == ERR_NULL, name
    for kw in (dict(rt=1), dict(rt=5), dict(scoring=2), dict(scoring=-1), dict(renorm=2)):
        assert call(**kw) == ERR_ARG, kw
    for kw in (dict(T=-1), dict(T=17), dict(E=0), dict(E=1025), dict(topk=0), dict(topk=9), dict(E=64, topk=33),
               dict(H=40), dict(H=0), dict(I=24), dict(I=0), dict(I=1 << 30)):
        assert call(**kw) == ERR_SHAPE, kw
    for kw in (dict(x=BASE[0] + 8), dict(r=BASE[1] + 2), dict(rt=0, r=BASE[1] + 1), dict(bias=BASE[2] + 2),
               dict(p13=BASE[3] + 8), dict(p2=BASE[6] + 8), dict(g13=BASE[5] + 2), dict(g2=BASE[8] + 1),
               dict(ws=BASE[9] + 8), dict(out=BASE[10] + 8), dict(ids=BASE[11] + 1), dict(w=BASE[12] + 2)):
        assert call(**kw) == ERR_ALIGN, kw
    for kw in (dict(out=BASE[0]), dict(ws=BASE[0] + 256), dict(out=BASE[9] + 256), dict(ids=BASE[12]),
               dict(ids=BASE[1]), dict(w=BASE[2] + 4), dict(out=BASE[4] - 16), dict(ws=BASE[6] + 16)):
        assert call(**kw) == ERR_ALIAS, kw
    assert call(T=0) == OK
    assert call(T=0, x=0, r=0, ws=0, out=0, ids=0, w=0, bias=0) == OK
    lib = B.load_library()
    assert lib.nvfp4_moe_decode_workspace_bytes(17, 2, 8, 512, 256) == 0
    assert lib.nvfp4_moe_decode_workspace_bytes(4, 9, 8, 512, 256) == 0
    assert lib.nvfp4_moe_decode_workspace_bytes(4, 2, 8, 512, 256) > 0


def test_binding_refusals():
    x = torch.zeros((1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):                      # not a device tensor
        B.nvfp4_moe_w4a16_decode(x, torch.zeros(1, 4), 2, (), ())
    with pytest.raises(B.NVFP4ShapeError):
        B.moe_decode_workspace(17, 2, 8, 512, 256, "cpu")


def test_routing_oracle_by_hand():
    ids, w = D.route(np.log([[1.0, 4.0, 4.0, 1.0]]), 3)
    assert ids.tolist() == [[1, 2, 0]] and np.allclose(w, [[4 / 9, 4 / 9, 1 / 9]])
    ids, w = D.route(np.log([[1.0, 4.0, 4.0, 1.0]]), 2, renormalize=False, weight_scale=2.0)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[0.8, 0.8]])
    ids, w = D.route([[0.0, -np.inf, np.nan, np.log(3.0)]], 3, "sigmoid", renormalize=False)
    assert ids.tolist() == [[3, 0, -1]] and np.allclose(w, [[0.75, 0.5, 0.0]])
    ids, w = D.route([[0.0, 0.0, 0.0]], 1, "sigmoid", bias=np.array([0.0, 0.1, 0.2]))
    assert ids.tolist() == [[2]] and np.allclose(w, [[1.0]])
    ids, w = D.route([[-np.inf, np.nan]], 2)
    assert ids.tolist() == [[-1, -1]] and w.tolist() == [[0.0, 0.0]]
