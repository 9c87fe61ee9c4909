"""GPU parity of nvfp4_moe_w4a16_decode with the float64 oracle: token counts
1 to 16, expert counts across the routing kernel's forms, ragged H and I, both
scorings, correction bias, ties, rows whose router leaves nothing, and graph
replays.  Chosen experts must be equal; weights and outputs lie within derived
bounds."""

import numpy as np
import pytest
import torch

import oracle.moe_decode_oracle as D
import oracle.nvfp4_moe_oracle as MO
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


@pytest.mark.parametrize("T,H,I", [(1, 64, 64), (3, 2048, 256), (16, 512, 288), (2, 1024, 4640), (5, 48, 272)])
def test_hidden_activations_keep_their_bits(T, H, I):
    """Pairs of nearly equal hidden activations against weights of opposite signs: the output is about
    2^-8 of its terms, and what the hidden activation loses in rounding shows in full.  Each token has
    two activations and each expert three pairs of columns, so no sum has more than a few terms: its
    float32 errors stay below 2^-18 of the terms, silu's and the routing weights' too, and the hidden
    activation may lose 2^-17 of itself."""
    E, cols = 2, np.array([0, I // 2 // 2 * 2, I - 2])
    rng = np.random.default_rng(T + I)
    code = lambda: rng.integers(1, 4, (E, 3)).astype(np.uint8) * 2         # 1, 2 or 4
    p13, p2 = np.zeros((E, 2 * I, H // 2), np.uint8), np.zeros((E, H, I // 2), np.uint8)
    k0, k1 = 6, H - 10                                   # even: low nibbles
    p13[:, cols, k0 // 2] = p13[:, cols + 1, k0 // 2] = code()             # w1: columns 2 j and 2 j + 1 alike
    p13[:, I + cols, k0 // 2] = p13[:, I + cols + 1, k0 // 2] = code()     # w3: but for its second term
    p13[:, I + cols, k1 // 2] = code()
    n = rng.integers(1, 8, (E, H, 3)).astype(np.uint8)
    p2[:, :, cols // 2] = n | ((n | 8) << 4)             # opposite signs
    s13, s2 = np.full((E, 2 * I, H // 16), 0x38, np.uint8), np.full((E, H, I // 16), 0x38, np.uint8)    # 1
    w13, w2 = (p13, s13, np.float32([0.5, 0.25])), (p2, s2, np.float32([0.5, 1.0]))
    x = np.zeros((T, H), np.float32)
    x[:, k0] = rng.uniform(0.5, 1.5, T)
    x[:, k1] = x[:, k0] * rng.uniform(0.5, 1.0, T) * 2.0 ** -8
    xb = torch.from_numpy(x).to(torch.bfloat16)
    x_bits = xb.view(torch.int16).numpy().view(np.uint16)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    out, ids, w = B.nvfp4_moe_w4a16_decode(xb.to(DEV), torch.from_numpy(logits).to(DEV), 2, upload(w13), upload(w2))
    torch.cuda.synchronize()
    want_ids, want_w = D.route(logits, 2)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    ref = MO.moe_ref(x_bits, want_ids, want_w.astype(np.float32), w13, w2)
    want, mag = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(2):
            e, a = want_ids[t, j], ref["a"][2 * t + j]
            want[t] += want_w[t, j] * (ref["w2deq"][e] @ a)
            mag[t] += want_w[t, j] * (np.abs(ref["w2deq"][e]) @ np.abs(a))
    err = np.abs(f64(out) - want)
    bound = mag * (2.0 ** -17 + 3 * 2.0 ** -18) + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7)
    assert np.all(mag > 0) and np.median(bound / np.abs(want)) < 0.05
    assert np.all(err <= bound), f"{(err > bound).mean():.3f} of the outputs, worst {(err / bound).max():.1f}"


def random_experts(E, N, K, seed):
    """Any codes, block scales of 0.25 to 1.875, global scales that keep outputs near 1."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    packed = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.int16).to(torch.uint8)
    scales = torch.randint(0x28, 0x40, (E, N, K // 16), generator=g, device=DEV, dtype=torch.int16).to(torch.uint8)
    return packed, scales, (0.5 + torch.rand((E,), generator=g, device=DEV)) * 0.5 / K ** 0.5


def dequant64(w, e):
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEV)
    p = w[0][e]
    codes = lut[torch.stack((p & 15, p >> 4), -1).int()].view(p.shape[0], -1, 16)
    return (codes * w[1][e].view(torch.float8_e4m3fn).double().unsqueeze(2)).view(p.shape[0], -1) * w[2][e].double()


@pytest.mark.parametrize("T,E,topk,H,I", [
    (16, 32, 4, 8192, 2400),       # two passes over H, and more units than the sums of one workgroup a unit hold
    (16, 24, 3, 4128, 4128),       # two passes over either
    (7, 256, 8, 5120, 512), (3, 60, 4, 7168, 2048), (16, 128, 8, 2048, 768)])
def test_many_experts(T, E, topk, H, I):
    """Sizes of real layers, in float64 on the device, with the oracle's bound."""
    w13, w2 = random_experts(E, 2 * I, H, 1), random_experts(E, H, I, 2)
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    router = torch.randn((T, E), generator=g, device=DEV)
    out, ids, w = B.nvfp4_moe_w4a16_decode(x, router, topk, w13, w2, scoring="sigmoid")
    want_ids, want_w = D.route(router.cpu().double().numpy(), topk, "sigmoid")
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    wt = torch.from_numpy(want_w).to(DEV)
    want, slack, u = torch.zeros((T, H), dtype=torch.float64, device=DEV), torch.zeros((T, H), dtype=torch.float64, device=DEV), D.U
    for e in sorted(set(want_ids.flatten())):
        t, j = (torch.from_numpy(a).to(DEV) for a in np.nonzero(want_ids == e))
        d13, d2, xe = dequant64(w13, e), dequant64(w2, e), x[t].double()
        h, dh = xe @ d13.t(), (H + 4) * 2 * u * (xe.abs() @ d13.abs().t())
        (gate, up), (dg, du) = h.split(I, 1), dh.split(I, 1)
        sg = torch.sigmoid(gate)
        a = gate * sg * up
        slope = (sg * (1 + gate * (1 - sg))).abs() + 0.1 * dg
        da = slope * up.abs() * dg + (gate * sg).abs() * du + dg * du + (2.0 ** -17 + 2.0 ** -20) * a.abs()
        mag = (a.abs() + da) @ d2.abs().t()
        wj = wt[t, j].unsqueeze(1)
        want.index_add_(0, t, wj * (a @ d2.t()))
        slack.index_add_(0, t, wj * (da @ d2.abs().t() + ((I + 8) * 2 + 48 + topk) * u * mag))
    err = (out.double() - want).abs()
    assert torch.all(err <= slack + 2.0 ** -8 * want.abs() * (1 + 2.0 ** -7)), (err / slack).max()
    # worst cases aside, an output is the nearest bf16 value or, where the sums' errors (about 2^-20 of
    # the terms' norm) cross a border, its neighbour: a twentieth at most
    assert (out != want.to(torch.bfloat16)).double().mean() < 0.05


@pytest.mark.parametrize("T,H,I", [(8, 512, 512), (3, 528, 272), (16, 1024, 256)])
def test_agrees_with_the_layer_over_given_ids_within_both_bounds(T, H, I):
    """nvfp4_moe_w4a16_forward on the routing reported here: apart by no more than the two bounds."""
    E, topk = 8, 2
    w13, w2 = experts(E, 2 * I, H, 5), experts(E, H, I, 6)
    x = wl.random_activation_bits(T, H, seed=5)
    router = torch.randn((T, E), generator=torch.Generator().manual_seed(T)).to(DEV)
    out, ids, w = B.nvfp4_moe_w4a16_decode(dev_bf16(x), router, topk, upload(w13), upload(w2))
    other = B.nvfp4_moe_w4a16_forward(dev_bf16(x), ids, w, upload(w13), upload(w2))
    hids, hw = ids.cpu().numpy(), w.cpu().numpy()
    _, bound = D.layer(x, hids, hw.astype(np.float64), w13, w2)
    tol = MO.moe_tolerance(MO.moe_ref(x, hids, hw, w13, w2), hw, H)
    assert np.all(np.abs(f64(out) - f64(other)) <= bound + tol)
