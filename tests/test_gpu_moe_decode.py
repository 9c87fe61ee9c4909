"""GPU parity of nvfp4_moe_w4a16_decode with the float64 oracle: token counts
1 to 16, expert counts across the routing kernel's forms, ragged H and I, both
scorings, correction bias, ties, rows whose router leaves nothing, and graph
replays.  Chosen experts must be equal; weights and outputs lie within derived
bounds."""

import numpy as np
import pytest
import torch

import oracle.moe_decode_oracle as D
from nvfp4_w4a16_lm_amd import binding as B
from nvfp4_w4a16_lm_amd import workloads as wl

from gpu_util import DEV, dev_bf16, host_bits
from test_gpu_graphs import capture
from test_gpu_moe import experts, f64, upload

pytestmark = pytest.mark.gpu


def check(T, E, topk, H, I, seed, scoring="softmax", renormalize=True, bias=None, weight_scale=1.0, logits=None,
          router_dtype=torch.float32):
    w13, w2 = experts(E, 2 * I, H, seed), experts(E, H, I, seed + 1)
    x = wl.random_activation_bits(T, H, seed=seed)
    rng = np.random.default_rng(seed)
    if logits is None:
        logits = 1.5 * rng.standard_normal((T, E))
    router = torch.from_numpy(np.asarray(logits, np.float32)).to(router_dtype).to(DEV)
    bd = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).to(DEV)
    out, ids, w = B.nvfp4_moe_w4a16_decode(dev_bf16(x), router, topk, upload(w13), upload(w2), scoring=scoring,
                                           renormalize=renormalize, correction_bias=bd, weight_scale=weight_scale)
    torch.cuda.synchronize()
    l64 = router.cpu().to(torch.float64).numpy()
    b64 = None if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    want_ids, want_w = D.route(l64, topk, scoring, renormalize, b64, weight_scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.all(np.abs(w.cpu().numpy() - want_w) <= 48 * D.U * np.abs(want_w))
    want, bound = D.layer(x, want_ids, want_w, w13, w2)
    err = np.abs(f64(out) - want)
    assert np.all(err <= bound), (np.argwhere(err > bound)[:4], err.max())
    return out, ids, w


@pytest.mark.parametrize("T,E,topk,H,I", [
    (1, 1, 1, 16, 16), (1, 8, 2, 512, 256), (2, 8, 2, 48, 272), (3, 4, 4, 272, 48), (16, 8, 2, 1024, 512),
    (5, 64, 6, 256, 128), (4, 65, 8, 128, 64), (7, 128, 8, 304, 80), (16, 256, 8, 64, 32), (2, 300, 10, 32, 48),
    (16, 1024, 3, 16, 16), (9, 32, 32, 64, 64), (16, 16, 16, 528, 1040), (1, 8, 2, 2048, 4096), (11, 3, 1, 4112, 256),
    # H and I multiples of 32: rows that end inside a chunk, one to several chunks and passes over K
    (2, 4, 2, 32, 32), (16, 8, 3, 96, 160), (5, 8, 2, 1056, 288), (3, 5, 2, 4128, 512), (2, 3, 2, 512, 4640),
    (4, 20, 4, 64, 8224), (7, 300, 6, 288, 96), (1, 2, 1, 8224, 64)])
def test_sizes(T, E, topk, H, I):
    check(T, E, topk, H, I, seed=T + E + topk + H + I)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_scorings(scoring, renormalize):
    check(6, 40, 5, 128, 96, 3, scoring, renormalize, weight_scale=2.5)
    # a bias far apart from expert to expert, so that rounding does not decide the choice
    bias = 0.03125 * np.random.default_rng(1).permutation(40)
    check(6, 40, 5, 128, 96, 4, scoring, renormalize, bias=bias)
    check(6, 40, 5, 128, 96, 5, scoring, renormalize, router_dtype=torch.bfloat16)


def test_ties_go_to_the_lower_expert():
    _, ids, w = check(3, 130, 4, 64, 32, 6, logits=np.zeros((3, 130)))
    assert ids.cpu().tolist() == [[0, 1, 2, 3]] * 3 and torch.all(w == 0.25)
    logits = np.zeros((2, 130))
    logits[:, [5, 70, 129]] = 2.0
    logits[1, 3] = -0.0
    _, ids, _ = check(2, 130, 4, 64, 32, 7, logits=logits)
    assert ids.cpu().tolist() == [[5, 70, 129, 0]] * 2


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_rows_with_few_or_no_experts(scoring):
    logits = np.random.default_rng(2).standard_normal((5, 10))
    logits[0] = -np.inf
    logits[1, 1:] = -np.inf
    logits[2, :5] = np.nan
    logits[3] = np.nan
    logits[4, 3] = np.finfo(np.float32).min
    out, ids, w = check(5, 10, 3, 64, 48, 8, scoring, logits=logits)
    assert ids[0].tolist() == [-1] * 3 and ids[3].tolist() == [-1] * 3 and not out[[0, 3]].any()
    assert ids[1].tolist() == [0, -1, -1] and w[1].tolist()[1:] == [0.0, 0.0]
    check(5, 10, 3, 64, 48, 9, scoring, logits=np.full((5, 10), -np.inf))


def test_optional_outputs_buffers_and_a_side_stream():
    T, E, topk, H, I = 3, 8, 2, 256, 128
    w13, w2 = upload(experts(E, 2 * I, H, 1)), upload(experts(E, H, I, 2))
    x = dev_bf16(wl.random_activation_bits(T, H, seed=1))
    router = torch.randn((T, E), device=DEV)
    want = B.nvfp4_moe_w4a16_decode(x, router, topk, w13, w2)
    ws = B.moe_decode_workspace(T, topk, E, H, I, DEV)
    ws.fill_(0xFF)                                       # the workspace needs no preparation
    guard = torch.full((T * H + 64,), 9.0, dtype=torch.bfloat16, device=DEV)
    out = guard[:T * H].view(T, H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = B.nvfp4_moe_w4a16_decode(x, router, topk, w13, w2, out=out, workspace=ws)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.all(guard[T * H:] == 9.0)
    lib = B.load_library()                               # without the routing outputs
    st = lib.nvfp4_moe_w4a16_decode(x.data_ptr(), T, H, router.data_ptr(), 2, E, topk, 0, 1, None, 1.0,
                                    *[t.data_ptr() for t in (*w13, *w2)], I, ws.data_ptr(), out.data_ptr(), None,
                                    None, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(out, want[0])
    assert B.nvfp4_moe_w4a16_decode(x[:0], router[:0], topk, w13, w2, workspace=ws)[0].shape == (0, H)


def test_same_routing_as_the_layer_over_given_ids():
    """The existing layer on the routing reported here gives the same output up to its own roundings."""
    T, E, topk, H, I = 8, 8, 2, 512, 512
    w13, w2 = upload(experts(E, 2 * I, H, 5)), upload(experts(E, H, I, 6))
    x = dev_bf16(wl.random_activation_bits(T, H, seed=5))
    out, ids, w = B.nvfp4_moe_w4a16_decode(x, torch.randn((T, E), device=DEV), topk, w13, w2)
    other = B.nvfp4_moe_w4a16_forward(x, ids, w, w13, w2)
    scale = out.float().abs().mean()
    assert (out.float() - other.float()).abs().max() <= 0.1 * scale


def test_infinite_activation_reaches_its_token_only():
    T, E, topk, H, I = 4, 8, 2, 128, 64
    w13, w2 = upload(experts(E, 2 * I, H, 7)), upload(experts(E, H, I, 8))
    x = dev_bf16(wl.random_activation_bits(T, H, seed=7))
    x[2, 5] = float("inf")
    out, _, _ = B.nvfp4_moe_w4a16_decode(x, torch.zeros((T, E), device=DEV), topk, w13, w2)
    assert not torch.isfinite(out[2]).all() and torch.isfinite(out[[0, 1, 3]]).all()


def test_graph_replays():
    T, E, topk, H, I = 4, 16, 4, 256, 128
    w13, w2 = upload(experts(E, 2 * I, H, 3)), upload(experts(E, H, I, 4))
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    router = torch.zeros((T, E), device=DEV)
    ws = B.moe_decode_workspace(T, topk, E, H, I, DEV)
    out = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    held = []
    graph = capture(lambda: held.append(B.nvfp4_moe_w4a16_decode(x, router, topk, w13, w2, out=out, workspace=ws)))
    _, ids, w = held[-1]
    for seed in (1, 2, 3):
        x.copy_(dev_bf16(wl.random_activation_bits(T, H, seed=seed)))
        router.copy_(torch.randn((T, E), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, ids, w)]
        for a, b in zip(got, B.nvfp4_moe_w4a16_decode(x, router, topk, w13, w2)):
            assert torch.equal(a, b), f"replay {seed}"
