"""The training example: every stage of its step against the float64 oracle on
the tensors that entered the stage, the served copies against the oracle of
theirs, and gradients and served copies captured into a graph and replayed."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle.dense_oracle as D
import oracle.nvfp4_oracle as O
from nvfp4_w4a16_lm_amd import binding as B

from gpu_util import DEV, host_bits
from test_gpu_graphs import capture

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "trained_head.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("trained_head", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def f64(t):
    return t.detach().cpu().double().numpy()


def within(got, want, bound):
    err = np.abs(f64(got) - want)
    assert np.all(err <= bound), (err.max(), (err / bound).max())


@pytest.mark.parametrize("tokens,vocab,hidden,inner", [(1, 300, 64, 128), (40, 1003, 256, 528), (300, 2000, 144, 272)])
def test_step_stage_by_stage(example, tokens, vocab, hidden, inner):
    a = example.inputs(tokens, vocab, hidden, inner, DEV, seed=tokens)
    a["targets"][0] = 7
    a["dloss"][0] = 1.0 / tokens
    w = {n: f64(a[n]) for n in ("x", "w13", "w2", "head", "dloss")}
    t = a["targets"].cpu().numpy().astype(np.int64)
    rate = 0.25
    g, logits, scored = example.step(**a, rate=rate)
    (y, h, act), (by, bh, ba) = D.gated_ffn(w["x"], w["w13"], w["w2"])
    within(g["kept"].h, h, bh)
    within(g["kept"].act, act, ba)
    total = w["x"] + y
    within(g["hidden"], total, by + D.HALF * (np.abs(total) + by))              # one more rounding: the residual's
    hid = f64(g["hidden"])
    loss, lse, bl, be = D.linear_ce(hid, w["head"], t)
    within(g["ce"].loss, loss, bl)
    within(g["ce"].lse, lse, be)
    (dh, dw, _), (bdh, bdw, _) = D.linear_ce_backward(hid, w["head"], t, w["dloss"])
    within(g["dhidden"], dh, bdh)
    within(g["dhead"], dw, bdw)
    (dx, d13, d2), (bx, b13, b2) = D.gated_ffn_backward(w["x"], f64(g["kept"].h), f64(g["kept"].act), w["w13"], w["w2"],
                                                                f64(g["dhidden"]))
    within(g["dw13"], d13, b13)
    within(g["dw2"], d2, b2)
    sum_dx = f64(g["dhidden"]) + dx
    within(g["dx"], sum_dx, bx + D.HALF * (np.abs(sum_dx) + bx))
    # the stepped head: one bf16 rounding of w - rate * dw; its served copies are those of the stepped bits
    within(a["head"], w["head"] - rate * f64(g["dhead"]), D.HALF * np.abs(w["head"] - rate * f64(g["dhead"])) + 2.0 ** -20)
    packed, scales, gs = O.quantize(host_bits(a["head"]))
    got = a["nvfp4_copy"]
    assert np.array_equal(got[0].cpu().numpy(), packed) and np.array_equal(got[1].view(torch.uint8).cpu().numpy(), scales)
    assert np.float32(got[2].item()) == gs
    wq, ws = D.int8_quantize_rows(f64(a["head"]))
    xq, xs = D.int8_quantize_rows(hid)
    ref, bound = D.int8_gemm(xq, xs, wq, ws)
    within(logits, ref, bound)
    lp = torch.log_softmax(logits.double(), 1).cpu()
    keep = torch.from_numpy(t >= 0)
    want = torch.where(keep, lp.gather(1, torch.from_numpy(np.maximum(t, 0)).unsqueeze(1)).squeeze(1), 0.0)
    assert torch.allclose(scored.token_logprobs.cpu().double(), want, atol=1e-4)


def test_graph_replays(example):
    a = example.inputs(40, 1003, 128, 272, DEV, seed=1)
    held = []

    def call():
        g = example.gradients(a["x"], a["w13"], a["w2"], a["head"], a["targets"], a["dloss"])
        logits, scored = example.served(g["hidden"], a["head"], a["nvfp4_copy"], a["targets"])
        return [g["dx"], g["dhead"], g["dw13"], g["dw2"], *g["ce"], logits, scored.token_logprobs, *a["nvfp4_copy"]]
    graph = capture(lambda: held.append(call()))
    for seed in (2, 3, 4):
        b = example.inputs(40, 1003, 128, 272, DEV, seed=seed)
        for n in ("x", "w13", "w2", "head", "targets", "dloss"):
            a[n].copy_(b[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held[-1]]
        for x, y in zip(got, call()):
            assert torch.equal(x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x,
                               y.view(torch.uint8) if y.dtype == torch.float8_e4m3fn else y)


def test_two_streams_and_workspaces_at_once(example):
    """Two steps in flight on two streams, each with its own workspace, equal the same steps alone."""
    runs = [example.inputs(70, 1500, 144, 272, DEV, seed=s) for s in (5, 6)]
    want = [example.gradients(*(r[n] for n in ("x", "w13", "w2", "head", "targets", "dloss"))) for r in runs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for r, s in zip(runs, streams):
        with torch.cuda.stream(s):
            got.append(example.gradients(*(r[n] for n in ("x", "w13", "w2", "head", "targets", "dloss"))))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for n in ("hidden", "dx", "dhead", "dw13", "dw2"):
            assert torch.equal(g[n], w[n]), n


def test_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["trained_head.py", "--tokens", "33", "--vocab", "500", "--hidden", "64"])
    example.main()
    assert capsys.readouterr().out.count("served in int8") == 3
