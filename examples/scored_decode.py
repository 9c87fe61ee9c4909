"""One decode step's tail, scored, and the gradient of a policy-gradient loss.

A batch of hidden states passes the expert layer from its router's logits
(nvfp4_moe_w4a16_decode), an int4 lm_head gives the logits (nvfp4_int4_gemm),
a grammar's mask and the sampling temperatures apply, and nvfp4_logprobs
reports each sampled token's log probability and rank, the entropy and the
best alternatives.  nvfp4_logprobs_backward then gives the gradient of
    loss = mean( -advantage * logprob - 0.01 * entropy )
with respect to the logits.  Weights are random; sizes are small by default.

    python examples/scored_decode.py [--tokens 8] [--vocab 32000] [--hidden 2048]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from nvfp4_w4a16_lm_amd import binding as B  # noqa: E402


def nvfp4_experts(e: int, n: int, k: int, gen: torch.Generator, dev) -> tuple:
    """Random NVFP4 expert weights, quantized one expert at a time by the library."""
    parts = [B.nvfp4_quantize((0.02 * torch.randn((n, k), generator=gen, device=dev)).to(torch.bfloat16))
             for _ in range(e)]
    return tuple(torch.stack([p[i].view(torch.uint8) if i == 1 else p[i] for p in parts]) for i in range(3))


def int4_head(vocab: int, k: int, group: int, gen: torch.Generator, dev) -> tuple:
    """A random lm_head in the int4 group layout: (packed int32 [N, K / 8], scales [N, K / group])."""
    w = 0.02 * torch.randn((vocab, k // group, group), generator=gen, device=dev)
    scales = (w.abs().amax(2) / 7.5).to(torch.bfloat16)
    codes = (torch.round(w / scales.float().unsqueeze(2)) + 8).clamp_(0, 15).to(torch.int64).view(vocab, k // 8, 8)
    words = (codes << (4 * torch.arange(8, device=dev))).sum(2)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32), scales


def allow(mask: torch.Tensor) -> torch.Tensor:
    """bool [M, V] -> the bit mask nvfp4_logprobs takes, int32 [M, ceil(V / 32)]."""
    m, v = mask.shape
    bits = torch.zeros((m, (v + 31) // 32 * 32), dtype=torch.int64, device=mask.device)
    bits[:, :v] = mask
    words = (bits.view(m, -1, 32) << torch.arange(32, device=mask.device)).sum(2)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def step(hidden, router, w13, w2, head, sampled, temperatures, allowed, advantage, experts_per_token=2, topk=5):
    """The tail of one decode step; everything stays on the device and the stream."""
    moe, ids, weights = B.nvfp4_moe_w4a16_decode(hidden, router, experts_per_token, w13, w2)
    hidden = hidden + moe
    logits = B.nvfp4_int4_gemm(hidden, *head)
    scored = B.nvfp4_logprobs(logits, sampled, topk=topk, temperatures=temperatures, allowed=allowed)
    m = logits.shape[0]
    dlogits = B.nvfp4_logprobs_backward(logits, sampled, scored.lse, scored.entropy, dlogprob=-advantage / m,
                                        dentropy=torch.full_like(advantage, -0.01 / m), temperatures=temperatures,
                                        allowed=allowed)
    return logits, ids, weights, scored, dlogits


def inputs(tokens: int, vocab: int, hidden: int, dev="cuda:0", experts: int = 8, inner: int = 1024, seed: int = 0):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    x = torch.randn((tokens, hidden), generator=gen, device=dev).to(torch.bfloat16)
    mask = torch.rand((tokens, vocab), generator=gen, device=dev) < 0.5
    sampled = torch.randint(0, vocab, (tokens,), generator=gen, device=dev)
    mask.scatter_(1, sampled.unsqueeze(1), True)
    return dict(hidden=x, router=torch.randn((tokens, experts), generator=gen, device=dev),
                w13=nvfp4_experts(experts, 2 * inner, hidden, gen, dev), w2=nvfp4_experts(experts, hidden, inner, gen, dev),
                head=int4_head(vocab, hidden, 128, gen, dev), sampled=sampled.to(torch.int32),
                temperatures=0.6 + 0.6 * torch.rand((tokens,), generator=gen, device=dev), allowed=allow(mask),
                advantage=torch.randn((tokens,), generator=gen, device=dev))


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=8)
    p.add_argument("--vocab", type=int, default=32000)
    p.add_argument("--hidden", type=int, default=2048)
    a = p.parse_args()
    _, ids, _, scored, dlogits = step(**inputs(a.tokens, a.vocab, a.hidden))
    for t in range(a.tokens):
        best = ", ".join(f"{i}: {lp:.3f}" for i, lp in zip(scored.top_ids[t].tolist(), scored.top_logprobs[t].tolist()))
        print(f"token {t}: experts {ids[t].tolist()}, logprob {float(scored.token_logprobs[t]):.3f} "
              f"(rank {int(scored.token_ranks[t])}), entropy {float(scored.entropy[t]):.3f}, best {best}")
    print(f"|dlogits| = {float(dlogits.float().norm()):.4e}")


if __name__ == "__main__":
    main()
