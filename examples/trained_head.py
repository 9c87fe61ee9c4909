"""One training step of a model's last block and its head, then the served copies.

Hidden states pass a gated feed-forward block (nvfp4_gated_ffn), the residual
is added, and nvfp4_linear_ce takes the cross entropy straight from the result
and the bf16 lm_head weight; nvfp4_linear_ce_backward and
nvfp4_gated_ffn_backward give the gradients, and plain SGD moves the weights.
The served copies follow the new head: nvfp4_refresh_inplace rewrites the NVFP4
one, nvfp4_int8_quantize_rows makes an int8 one, and nvfp4_int8_gemm with
nvfp4_logprobs scores the same targets from it.  Weights are random; sizes are
small by default.

    python examples/trained_head.py [--tokens 256] [--vocab 8000] [--hidden 512]
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


def gradients(x, w13, w2, head, targets, dloss):
    """Loss and gradients of block, residual and head; everything stays on the device and the stream."""
    y, kept = B.nvfp4_gated_ffn(x, w13, w2, keep_h=True)
    hidden = x + y
    ce = B.nvfp4_linear_ce(hidden, head, targets)
    dhidden, dhead, _ = B.nvfp4_linear_ce_backward(hidden, head, targets, ce.stats, dloss)
    dx, dw13, dw2 = B.nvfp4_gated_ffn_backward(x, kept, w13, w2, dhidden)
    return dict(hidden=hidden, kept=kept, ce=ce, dhidden=dhidden, dhead=dhead, dx=dhidden + dx, dw13=dw13, dw2=dw2)


def served(hidden, head, nvfp4_copy, targets):
    """The head's served copies, and the targets' log probabilities from the int8 one."""
    B.nvfp4_refresh_inplace(head, *nvfp4_copy)
    wq, ws = B.nvfp4_int8_quantize_rows(head)
    xq, xs = B.nvfp4_int8_quantize_rows(hidden)
    logits = B.nvfp4_int8_gemm(xq, xs, wq, ws)
    return logits, B.nvfp4_logprobs(logits, targets)


def step(x, w13, w2, head, targets, dloss, nvfp4_copy, rate=0.5):
    g = gradients(x, w13, w2, head, targets, dloss)
    for w, d in ((head, g["dhead"]), (w13, g["dw13"]), (w2, g["dw2"])):
        w.add_(d, alpha=-rate)
    logits, scored = served(g["hidden"], head, nvfp4_copy, targets)
    return g, logits, scored


def inputs(tokens: int, vocab: int, hidden: int, inner: int, dev="cuda:0", seed: int = 0):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rand = lambda *s, std=1.0: (std * torch.randn(s, generator=gen, device=dev)).to(torch.bfloat16)
    targets = torch.randint(0, vocab, (tokens,), generator=gen, device=dev).to(torch.int32)
    targets[torch.rand((tokens,), generator=gen, device=dev) < 0.1] = -100          # padding
    counts = (targets >= 0).float()
    head = rand(vocab, hidden, std=hidden ** -0.5)
    return dict(x=rand(tokens, hidden), w13=rand(2 * inner, hidden, std=hidden ** -0.5),
                w2=rand(hidden, inner, std=inner ** -0.5), head=head, targets=targets, dloss=counts / counts.sum(),
                nvfp4_copy=B.nvfp4_quantize(head))


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=256)
    p.add_argument("--vocab", type=int, default=8000)
    p.add_argument("--hidden", type=int, default=512)
    a = p.parse_args()
    args = inputs(a.tokens, a.vocab, a.hidden, 4 * a.hidden)
    for i in range(3):
        g, _, scored = step(**args)
        loss = float((g["ce"].loss * args["dloss"]).sum())
        served_loss = float(-(scored.token_logprobs * args["dloss"]).sum())
        print(f"step {i}: loss {loss:.4f}; with the stepped head, served in int8: {served_loss:.4f}")


if __name__ == "__main__":
    main()
