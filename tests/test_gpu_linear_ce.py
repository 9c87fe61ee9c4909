"""GPU parity of the linear cross entropy and its gradients with the float64
oracle: sizes around every tile width and piece, rows that do not count (and
hold NaN), masked tokens, large logits, differences, outputs written exactly,
graph replays, given streams and shared workspaces."""

import numpy as np
import pytest
import torch

import oracle.dense_oracle as D
from nvfp4_w4a16_lm_amd import binding as B

from gpu_util import DEV
from test_boundary_dense import shared_targets, tied_targets
from test_gpu_graphs import capture

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def bf16(rng, *shape, sigma=1.0):
    return torch.from_numpy(sigma * rng.standard_normal(shape)).to(BF16)


def make(m, v, k, seed, bias=False, gone=0.0, sigma=1.0):
    rng = np.random.default_rng(seed)
    w = bf16(rng, v, k, sigma=1.3 / np.sqrt(k))
    t = rng.integers(0, v, m)
    x = bf16(rng, m, k, sigma=sigma) + torch.where(torch.from_numpy(rng.random((m, 1)) < 0.6), 6.0, 0.0).to(BF16) * w[t]
    t = np.where(rng.random(m) < gone, rng.choice([-100, -1, v, 2 ** 31 - 1], m), t)
    return dict(x=x.to(BF16), w=w, t=torch.from_numpy(t.astype(np.int32)), bias=bf16(rng, v) if bias else None,
                dloss=torch.from_numpy(rng.standard_normal(m).astype(np.float32) / m),
                dlse=torch.from_numpy(0.1 * rng.standard_normal(m).astype(np.float32) / m))


def dev(a):
    return {n: None if t is None else t.to(DEV) for n, t in a.items()}


def f64(t):
    return None if t is None else t.cpu().double().numpy()


def within(got, want, bound, what):
    got = f64(got)
    both = np.isfinite(want)
    assert np.array_equal(got[~both], want[~both], equal_nan=True), what
    err = np.abs(got[both] - want[both])
    assert np.all(err <= bound[both]), (what, err.max(), (err / bound[both]).max())


def forward(d, **kw):
    return B.nvfp4_linear_ce(d["x"], d["w"], d["t"], bias=d["bias"], **kw)


def backward(d, stats, dlse=True, **kw):
    return B.nvfp4_linear_ce_backward(d["x"], d["w"], d["t"], stats, d["dloss"], bias=d["bias"],
                                      dlse=d["dlse"] if dlse else None, **kw)


def check(a, dlse=True):
    d = dev(a)
    r = forward(d)
    n = {k: f64(t) for k, t in a.items()}
    t = a["t"].numpy().astype(np.int64)
    loss, lse, bl, be = D.linear_ce(n["x"], n["w"], t, n["bias"])
    within(r.loss, loss, bl, "loss")
    within(r.lse, lse, be, "lse")
    got = backward(d, r.stats, dlse)
    want, bounds = D.linear_ce_backward(n["x"], n["w"], t, n["dloss"], n["dlse"] if dlse else None, n["bias"])
    for g, y, b, what in zip(got, want, bounds, ("dx", "dw", "db")):
        if g is not None:
            within(g, y, b, what)
    assert (got[2] is None) == (a["bias"] is None)
    return d, r, got


@pytest.mark.parametrize("m,v,k", [
    (1, 1, 16), (1, 300, 48), (2, 257, 16), (5, 1003, 528), (17, 513, 144), (31, 700, 112), (32, 256, 256), (33, 255, 80),
    (63, 1003, 272), (65, 300, 1040), (127, 511, 64), (128, 515, 336), (129, 1003, 528), (200, 2003, 272), (257, 770, 144),
    (333, 3003, 528), (513, 300, 528), (3, 20011, 64)])
@pytest.mark.parametrize("full", [False, True])
def test_sizes(m, v, k, full):
    check(make(m, v, k, seed=m + v + k, bias=full, gone=0.3 if full else 0.0), dlse=full)


@pytest.mark.parametrize("m,v,k", [(333, 22003, 208), (700, 30003, 272), (400, 8000, 4096), (1100, 9000, 144)])
def test_wide_tiles(m, v, k):
    """Sizes at which the widest tiles are taken: 192 and 256 rows of logits, 256 of the weight's gradient."""
    check(make(m, v, k, seed=m, gone=0.1))


def test_several_pieces():
    """Enough rows that the vocabulary is taken in pieces, the last one ragged."""
    m, v, k = 40000, 4003, 32
    assert int(B.load_library().nvfp4_linear_ce_workspace_bytes(m, v, k, 1)) < 2 * m * v + 8 * m * k
    check(make(m, v, k, seed=3, bias=True, gone=0.05))


@pytest.mark.parametrize("m,v,k", [(3, 265795, 16), (1500, 50003, 32)])
def test_several_pieces_with_a_split_gradient_of_x(m, v, k):
    """Two pieces of the vocabulary, dx cut into parts (64 of 3 rows, 40 of 1500) that both pieces add to; the second
    piece is narrower, so that it leaves the last part as the first one made it."""
    a = make(m, v, k, seed=m, bias=True, gone=0.0 if m < 10 else 0.1)
    a["t"][:3] = torch.tensor([5, v // 2 + 1000, v - 1], dtype=torch.int32)
    check(a)


@pytest.mark.parametrize("m,v,k", [(5, 300, 16), (20, 1003, 64), (130, 1003, 16), (333, 3003, 528), (700, 2003, 144),
                                   (140, 300003, 16)])
def test_bias_gradient_takes_the_targets_unrounded(m, v, k):
    """Rows that share a few targets, again in other groups of rows and in both pieces of a wide vocabulary, with dz
    that add up to about nothing: what rounding takes from them is several times the bound of their sum."""
    x, w, bias, t, dloss = (torch.from_numpy(n) for n in shared_targets(m, v, k, seed=m))
    check(dict(x=x.to(BF16), w=w.to(BF16), bias=bias.to(BF16), t=t.to(torch.int32), dloss=dloss.float(), dlse=None),
          dlse=False)


@pytest.mark.parametrize("m,v,k", [(1, 1003, 64), (5, 300, 16), (20, 1003, 64), (40, 300003, 16), (130, 4003, 16), (333, 22003, 208),
                                   (700, 6003, 144), (1100, 9000, 144), (8500, 9003, 16)])
def test_gradients_take_the_targets_unrounded(m, v, k):
    """Rows of a target share their x, and their dz at it add up to about nothing: what rounding takes from them is
    several times the bounds of dx and of the target's row of dweight.  One to some thousand rows a target, in both pieces of
    a wide vocabulary, in every tile of the logits and of the weight's gradient."""
    x, w, bias, t, dloss = (torch.from_numpy(n) for n in tied_targets(m, v, k, seed=m))
    check(dict(x=x.to(BF16), w=w.to(BF16), bias=bias.to(BF16), t=t.to(torch.int32), dloss=dloss.float(), dlse=None),
          dlse=False)


@pytest.mark.parametrize("m", [150, 4000])
def test_one_target_for_all_rows(m):
    a = make(m, 1003, 144, seed=m, bias=True)
    a["t"][:] = 700
    a["t"][:m // 3] = -1
    check(a)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_rows_that_do_not_count_are_not_looked_at(m):
    a = make(m, 700, 144, seed=m, gone=0.4)
    a["t"][0] = -1
    d = dev(a)
    r = forward(d)
    want = backward(d, r.stats)
    gone = ((d["t"] < 0) | (d["t"] >= 700))
    for bad in (float("nan"), float("inf")):
        d["x"][gone] = bad
        d["dloss"][gone] = bad
        d["dlse"][gone] = bad
        r2 = forward(d)
        got = backward(d, r2.stats)
        assert all(torch.equal(p, q) for p, q in zip(r, r2))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.all(r.loss[gone] == 0) and torch.all(r.lse[gone] == 0) and torch.all(want[0][gone] == 0)
    assert torch.equal(r.stats[gone], torch.tensor([0.0, 1.0], device=DEV).expand(int(gone.sum()), 2))


@pytest.mark.parametrize("m", [3, 200])
def test_no_row_counts(m):
    a = make(m, 515, 64, seed=4, bias=True)
    a["t"][:] = -100
    d, r, (dx, dw, db) = check(a)
    assert not r.loss.any() and not dx.any() and not dw.any() and not db.any()


@pytest.mark.parametrize("m", [5, 150])
def test_masked_tokens(m):
    """A bias of -inf masks tokens: no probability, no gradient; whole tiles of them; a target among them; all."""
    a = make(m, 1003, 144, seed=6, bias=True)
    a["bias"][:300] = -float("inf")
    a["bias"][999] = -float("inf")
    a["t"][:3] = torch.tensor([5, 400, 999])
    d, r, (dx, dw, db) = check(a)
    assert float(r.loss[0]) == float("inf") and torch.isfinite(dx).all()
    assert not dw[:300].any() and not db[:300].any()
    a["bias"][:] = -float("inf")
    d = dev(a)
    r = forward(d)
    assert torch.all(r.lse == -float("inf")) and torch.all(r.loss == float("inf"))
    assert all(not t.any() for t in backward(d, r.stats))


def test_lowest_value_masks():
    """Biases of bfloat16's lowest value leave the others' probabilities as they are."""
    a = make(9, 600, 64, seed=8, bias=True)
    a["bias"][100:580] = torch.finfo(BF16).min
    a["t"] = torch.arange(9, dtype=torch.int32)
    check(a)


def test_large_logits_keep_their_accuracy():
    """Logits of thousands: p is taken relative to the row's maximum, not from a rounded lse."""
    for m in (4, 150):
        check(make(m, 700, 64, seed=11, sigma=3000.0))
    a = make(4, 700, 64, seed=12)
    a["bias"] = torch.full((700,), 2.0 ** 20, dtype=BF16)      # every logit near 2^20: steps of 2^-4
    d = dev(a)
    r = forward(d)
    dx, dw, db = backward(d, r.stats, dlse=False)
    s = db.double().sum() / d["dloss"].double().abs().sum()
    assert abs(float(s)) < 2.0 ** -6                            # p sums to one: dz over the vocabulary to zero


def test_infinite_and_nan_logits_stay_in_their_row():
    a = make(40, 700, 64, seed=13)
    a["x"][3, 5] = float("inf")
    a["x"][7, 9] = float("nan")
    d = dev(a)
    r = forward(d)
    bad = torch.zeros(40, dtype=torch.bool, device=DEV)
    bad[[3, 7]] = True
    assert torch.isnan(r.loss[bad]).all() and torch.isnan(r.lse[bad]).all()
    assert torch.isfinite(r.loss[~bad]).all()
    dx, _, _ = backward(d, r.stats)
    assert torch.isfinite(dx[~bad]).all() and torch.isnan(dx[bad]).any(1).all()


def test_a_target_whose_dz_rounds_to_infinity():
    """The gradient of the bias is then the infinity, without a remainder that would make it NaN.  bfloat16 takes what is
    past 2^128 (1 - 2^-9) to infinity; the largest dloss less its part p is."""
    a = make(1, 300, 64, seed=19, bias=True)
    t, top = int(a["t"][0]), float(torch.finfo(torch.float32).max)
    a["dloss"][:] = top
    a["bias"][t] = -32.0
    n = {k: f64(v) for k, v in a.items()}
    loss = D.linear_ce(n["x"], n["w"], np.array([t]), n["bias"])[0][0]
    assert top * (1 - np.exp(-loss)) > 2.0 ** 128 * (1 - 2.0 ** -10)
    d = dev(a)
    _, _, db = backward(d, forward(d).stats, dlse=False)
    assert float(db[t]) == -float("inf") and torch.isfinite(torch.cat((db[:t], db[t + 1:]))).all()


def test_gradient_against_differences():
    """The gradients along a direction against central differences of the oracle's loss."""
    a = make(20, 300, 64, seed=14, bias=True, gone=0.2)
    d, r, grads = check(a)
    n = {k: f64(t) for k, t in a.items()}
    t = a["t"].numpy().astype(np.int64)
    _, bounds = D.linear_ce_backward(n["x"], n["w"], t, n["dloss"], n["dlse"], n["bias"])

    def f(x, w, b):
        loss, lse, _, _ = D.linear_ce(x, w, t, b)
        return loss @ n["dloss"] + lse @ n["dlse"]
    rng = np.random.default_rng(1)
    for which, (grad, bound) in enumerate(zip(grads, bounds)):
        args = [n["x"], n["w"], n["bias"]]
        e = rng.standard_normal(args[which].shape)
        up, down = list(args), list(args)
        up[which], down[which] = args[which] + 1e-4 * e, args[which] - 1e-4 * e
        diff = (f(*up) - f(*down)) / 2e-4
        assert abs(diff - (f64(grad) * e).sum()) <= (bound * np.abs(e)).sum() + 1e-6


def test_buffers_are_written_exactly():
    """Through the C entry points: guards behind every output, optional outputs left out, workspace of stale NaN."""
    lib = B.load_library()
    m, v, k = 45, 515, 80
    d = dev(make(m, v, k, seed=15, bias=True, gone=0.2))
    r = forward(d)
    want = backward(d, r.stats)
    size = int(lib.nvfp4_linear_ce_workspace_bytes(m, v, k, 1))
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    outs = [torch.full((n + 32,), 3.0, dtype=dt, device=DEV)
            for n, dt in ((m, torch.float32), (2 * m, torch.float32), (m * k, BF16), (v * k, BF16), (v, BF16))]
    p = [t.data_ptr() for t in outs]
    q = {n: t.data_ptr() for n, t in d.items()}
    s = torch.cuda.current_stream().cuda_stream
    assert lib.nvfp4_linear_ce(q["x"], m, k, q["w"], v, q["bias"], q["t"], ws.data_ptr(), p[0], None, p[1], s) == 0
    assert lib.nvfp4_linear_ce_backward(q["x"], m, k, q["w"], v, q["bias"], q["t"], p[1], q["dloss"], q["dlse"],
                                        ws.data_ptr(), p[2], p[3], p[4], s) == 0
    torch.cuda.synchronize()
    for got, ref in zip(outs, (r.loss, r.stats, *want)):
        assert torch.equal(got[:ref.numel()], ref.flatten()) and torch.all(got[ref.numel():] == 3.0)
    assert torch.all(ws[size:] == 0xFF)
    for keep in range(3):                                # each gradient alone
        alone = [torch.full_like(t, 3.0) for t in outs[2:]]
        a = [t.data_ptr() if i == keep else None for i, t in enumerate(alone)]
        assert lib.nvfp4_linear_ce_backward(q["x"], m, k, q["w"], v, q["bias"], q["t"], p[1], q["dloss"], q["dlse"],
                                            ws.data_ptr(), *a, s) == 0
        torch.cuda.synchronize()
        for i, t in enumerate(alone):
            assert torch.equal(t, outs[2 + i]) if i == keep else torch.all(t == 3.0)


@pytest.mark.parametrize("m", [7, 150])
def test_graph_replays(m):
    d = dev(make(m, 1003, 144, seed=m, bias=True, gone=0.2))
    ws = B.linear_ce_workspace(m, 1003, 144, DEV)
    held = []

    def call():
        r = forward(d, workspace=ws)
        return (*r, *backward(d, r.stats, workspace=ws))
    graph = capture(lambda: held.append(call()))
    for seed in range(3):
        e = dev(make(m, 1003, 144, seed=50 + seed, bias=True, gone=0.3))
        for n in d:
            d[n].copy_(e[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held[-1]]
        for x, y in zip(got, call()):                    # another count of rows in every replay
            assert torch.equal(x, y)


def test_given_stream_and_small_workspace():
    d = dev(make(33, 700, 96, seed=21, gone=0.2))
    want = forward(d)
    grads = backward(d, want.stats)
    wide = dict(d, x=torch.stack([d["x"], d["x"]], -1)[..., 0], w=torch.stack([d["w"], d["w"]], -1)[..., 0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    r = forward(wide, stream=side)
    g = backward(wide, r.stats, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*r, *g[:2]), (*want, *grads[:2])))
    with pytest.raises(ValueError):
        forward(d, workspace=torch.empty((64,), dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        backward(d, want.stats, workspace=B.linear_ce_workspace(33, 700, 96, DEV, backward=False)[:64])


def test_workspace_kept_for_the_largest_batch():
    """One workspace of the largest batch, for every smaller one: the results are those of a fresh one."""
    v, k = 2003, 144
    ws = B.linear_ce_workspace(1025, v, k, DEV)
    for m in (1025, 1024, 513, 257, 256, 129, 128, 65, 64, 33, 32, 1):
        d = dev(make(m, v, k, seed=m, gone=0.1))
        r = forward(d)
        want = (*r, *backward(d, r.stats)[:2])
        s = forward(d, workspace=ws)
        got = (*s, *backward(d, s.stats, workspace=ws)[:2])
        assert all(torch.equal(x, y) for x, y in zip(got, want)), m


@pytest.mark.parametrize("m", [3, 200])
def test_gradients_left_out_and_given_buffers(m):
    """Every choice of gradients through the binding: those left out are None, the others are what they are together,
    made or in the caller's buffers; of an empty batch a buffer becomes zero."""
    d = dev(make(m, 515, 80, seed=m, bias=True, gone=0.2))
    stats = forward(d).stats
    want = backward(d, stats)
    names = ("dx", "dweight", "dbias")
    for mask in range(8):
        got = backward(d, stats, **{n: bool(mask >> i & 1) for i, n in enumerate(names)})
        assert all(torch.equal(g, w) if mask >> i & 1 else g is None for i, (g, w) in enumerate(zip(got, want)))
    bufs = [torch.full_like(t, 3.0) for t in want]
    got = backward(d, stats, **dict(zip(names, bufs)))
    assert all(g is b and torch.equal(g, w) for g, b, w in zip(got, bufs, want))
    plain = backward(dict(d, bias=None), stats, dx=False, dweight=False)
    assert plain == (None, None, None)                   # without a bias there is no dbias, unless a buffer asks for it
    db = backward(dict(d, bias=None), forward(dict(d, bias=None)).stats, dx=False, dweight=False, dbias=bufs[2])[2]
    assert db is bufs[2] and torch.isfinite(db).all()
    side = torch.cuda.Stream()
    bufs[0].fill_(3.0)
    torch.cuda.synchronize()
    got = backward(d, stats, stream=side, dweight=False, dx=bufs[0])
    side.synchronize()
    assert got[0] is bufs[0] and got[1] is None and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    empty = {n: t if n in ("w", "bias") else t[:0] for n, t in d.items()}
    dx, dw, db = backward(empty, stats[:0], dx=False, dweight=bufs[1].fill_(3.0))
    assert dx is None and dw is bufs[1] and not dw.any() and not db.any()
    for bad in (dict(dx=bufs[0][:-1]), dict(dweight=bufs[1].float()), dict(dbias=bufs[2].cpu())):
        with pytest.raises(ValueError):
            backward(d, stats, **bad)


def test_empty_batch():
    d = dev(make(2, 100, 32, seed=1, bias=True))
    e = {n: t if n in ("w", "bias") else t[:0] for n, t in d.items()}
    r = forward(e)
    assert r.loss.shape == (0,) and r.stats.shape == (0, 2)
    dx, dw, db = backward(e, r.stats)
    assert dx.shape == (0, 32) and not dw.any() and not db.any()


def test_binding_refusals():
    d = dev(make(4, 100, 32, seed=1))
    r = forward(d)
    for kw in (dict(t=d["t"].long()), dict(t=d["t"][:3]), dict(w=d["w"][:, :16].contiguous()),
               dict(bias=torch.zeros(99, dtype=BF16, device=DEV)), dict(bias=torch.zeros(100, device=DEV))):
        with pytest.raises(ValueError):
            forward({**d, **kw})
    with pytest.raises(ValueError):
        backward(d, r.stats[:, 0])
    with pytest.raises(ValueError):
        backward(dict(d, dloss=d["dloss"].double()), r.stats)
    with pytest.raises(B.NVFP4ShapeError):
        B.nvfp4_linear_ce(torch.zeros((4, 24), dtype=BF16, device=DEV), torch.zeros((9, 24), dtype=BF16, device=DEV),
                          d["t"])
