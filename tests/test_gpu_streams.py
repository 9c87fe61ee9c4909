"""Calls given a stream that is not the current one.  What a call copies or
allocates by itself is on the stream that it was given: the current stream is
kept busy meanwhile, so that a dense copy of an input made there would come
too late, and takes and overwrites memory straight after the call, so that a
temporary from its own pool would be lost.  Results must equal those of the
same call on the current stream."""

import pytest
import torch

from nvfp4_w4a16_lm_amd import binding as B
from nvfp4_w4a16_lm_amd import workloads as wl

from gpu_util import DEV, dev_bf16
from test_gpu_moe import experts, upload

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def wide(t):
    """The same values with columns apart: the call has to make its own dense copy."""
    return torch.stack([t, t], -1)[..., 0]


def bf16(*shape, seed=1, sigma=1.0):
    return (sigma * torch.randn(shape, generator=gen(seed), device=DEV)).to(BF16)


def moe_sizes():
    return 8, 8, 2, 256, 128                             # T, E, topk, H, I


def calls():
    """name -> (call, its inputs)"""
    T, E, k, H, I = moe_sizes()
    w13, w2 = upload(experts(E, 2 * I, H, 1)), upload(experts(E, H, I, 2))
    x = wide(dev_bf16(wl.random_activation_bits(T, H, seed=1)))
    router = torch.randn((T, E), generator=gen(2), device=DEV)
    ids = wide(torch.randint(0, E, (T, k), generator=gen(3), device=DEV, dtype=I32))
    w = wide(torch.rand((T, k), generator=gen(4), device=DEV))
    head = B.nvfp4_quantize(bf16(515, 256, sigma=0.02))
    gs = torch.tensor(0.01, device=DEV)
    xp, xs = B.nvfp4_quantize_activations(bf16(5, 256), gs)
    codes = torch.randint(-2 ** 31, 2 ** 31, (515, 32), generator=gen(5), device=DEV, dtype=torch.int64).to(I32)
    scales = (0.01 * torch.rand((515, 8), generator=gen(6), device=DEV)).to(BF16)
    logits = bf16(4, 20011, sigma=3.0)
    tok = torch.tensor([3, 2, 1, 0], dtype=I32, device=DEV)
    f = B.nvfp4_logprobs(logits, tok)
    one = torch.ones((4,), device=DEV)
    return {
        "quantize": (B.nvfp4_quantize, (wide(bf16(33, 64)),)),
        "w4a16_gemm": (B.nvfp4_w4a16_gemm, (x, *head)),
        "fp8_quantize_rows": (B.nvfp4_fp8_quantize_rows, (wide(bf16(33, 64)),)),
        "quantize_activations": (B.nvfp4_quantize_activations, (wide(bf16(33, 64)), gs)),
        "w4a4_gemm": (B.nvfp4_w4a4_gemm, (xp, xs, gs, *head)),
        "moe_gemm": (B.nvfp4_moe_w4a16_gemm, (x, ids, k, *w13)),
        "moe_silu_and_mul": (B.nvfp4_moe_silu_and_mul, (x,)),
        "moe_combine": (B.nvfp4_moe_combine, (wide(bf16(T * k, H)), w)),
        "moe_forward": (B.nvfp4_moe_w4a16_forward, (x, ids, w, w13, w2)),
        "moe_decode": (B.nvfp4_moe_w4a16_decode, (x, router, k, w13, w2)),
        "int4_gemm": (B.nvfp4_int4_gemm, (x, codes, scales)),
        "logprobs": (B.nvfp4_logprobs, (logits, tok, 5)),
        "logprobs_backward": (B.nvfp4_logprobs_backward, (logits, tok, f.lse, f.entropy, one, one)),
    }


def tensors(result):
    """A call's outputs as bytes (its workspace aside)."""
    out = result[:6] if isinstance(result, B.Logprobs) else result if isinstance(result, tuple) else (result,)
    return [t.contiguous().view(-1).view(torch.uint8) for t in out]


NAMES = ("quantize", "w4a16_gemm", "fp8_quantize_rows", "quantize_activations", "w4a4_gemm", "moe_gemm", "moe_silu_and_mul",
         "moe_combine", "moe_forward", "moe_decode", "int4_gemm", "logprobs", "logprobs_backward")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("raw", [False, True])
def test_given_stream(name, raw):
    call, args = calls()[name]
    want = [t.clone() for t in tensors(call(*args))]
    busy = torch.ones((4096, 4096), dtype=BF16, device=DEV)
    sink = torch.empty_like(busy)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(20):
            torch.mm(busy, busy, out=sink)               # some milliseconds on the current stream
        got = call(*args, stream=side.cuda_stream if raw else side)
        taken = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV)      # allocated at once, written behind the products
                 for n in (512, 4096, 1 << 16, 1 << 20) for _ in range(8)]
        side.synchronize()
        for a, b in zip(tensors(got), want):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
        for a, b in zip(tensors(got), want):
            assert torch.equal(a, b)
        del taken


@pytest.mark.parametrize("name", NAMES)
def test_allocations_are_on_the_given_stream(name, monkeypatch):
    call, args = calls()[name]
    seen, real = [], torch.empty

    def spy(*a, **k):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return real(*a, **k)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", spy)
    call(*args, stream=side)
    assert seen and set(seen) == {side.cuda_stream}
    seen.clear()
    call(*args, stream=0)                                # the raw handle of the default stream
    assert seen and set(seen) == {torch.cuda.default_stream().cuda_stream}
    torch.cuda.synchronize()
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_given_buffers_on_a_given_stream():
    T, E, k, H, I = moe_sizes()
    call, args = calls()["moe_decode"]
    want = [t.clone() for t in call(*args)]
    ws, out = B.moe_decode_workspace(T, k, E, H, I, DEV), torch.empty((T, H), dtype=BF16, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(*args, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert got[0] is out and all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_are_the_same_with_a_stream():
    with pytest.raises(ValueError):
        B.nvfp4_int4_gemm(torch.zeros((1, 64), dtype=BF16), torch.zeros((4, 8), dtype=I32), torch.zeros((4, 2), dtype=BF16),
                          stream=torch.cuda.Stream())
    with pytest.raises(B.NVFP4ShapeError):
        B.nvfp4_logprobs(torch.zeros((2, 9), device=DEV), topk=65, stream=torch.cuda.Stream())
