"""The decode-tail example: its four calls together against torch on the same
tensors, and the whole step captured into a graph and replayed."""

import importlib.util
import os

import pytest
import torch

from gpu_util import DEV
from test_gpu_graphs import capture

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "scored_decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("scored_decode", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,vocab,hidden", [(1, 1000, 256), (8, 32000, 512), (16, 5003, 1024)])
def test_step_agrees_with_torch(example, tokens, vocab, hidden):
    a = example.inputs(tokens, vocab, hidden, DEV, inner=256, seed=tokens)
    logits, ids, weights, scored, dlogits = example.step(**a)
    assert torch.allclose(weights.sum(1), torch.ones(tokens, device=DEV), atol=1e-6)
    assert torch.equal(ids, torch.topk(a["router"], 2, dim=1).indices.to(torch.int32))
    # log probabilities, entropy and gradient of the same logits by autograd in float64
    bits = (a["allowed"].unsqueeze(2) >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
    allowed = bits.flatten(1)[:, :vocab] == 1
    z = logits.detach().double().requires_grad_()
    logp = torch.log_softmax(z.masked_fill(~allowed, -1e300) / a["temperatures"].double().unsqueeze(1), 1)
    lp = logp.gather(1, a["sampled"].long().unsqueeze(1)).squeeze(1)
    entropy = -(logp.exp() * logp.masked_fill(~allowed, 0.0)).sum(1)
    assert torch.allclose(scored.token_logprobs.double(), lp, atol=1e-4)
    assert torch.allclose(scored.entropy.double(), entropy, atol=1e-4)
    (-(a["advantage"].double() * lp).mean() - 0.01 * entropy.mean()).backward()
    err = (dlogits.double() - z.grad).abs()
    assert torch.all(err <= 2.0 ** -8 * z.grad.abs() + 1e-5 * z.grad.abs().amax(1, keepdim=True))


def test_step_graph_replays(example):
    a = example.inputs(4, 4099, 512, DEV, inner=128, seed=5)
    held = []
    graph = capture(lambda: held.append(example.step(**a)))
    logits, ids, weights, scored, dlogits = held[-1]
    for seed in (1, 2, 3):
        a["hidden"].copy_(torch.randn((4, 512), generator=torch.Generator().manual_seed(seed)))
        a["router"].copy_(torch.randn((4, 8), generator=torch.Generator().manual_seed(seed + 9)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (logits, ids, weights, *scored[:6], dlogits)]
        l2, i2, w2, s2, d2 = example.step(**a)
        for x, y in zip(got, (l2, i2, w2, *s2[:6], d2)):
            assert torch.equal(x, y), f"replay {seed}"
