"""moe_balance_loss against the oracle's fp64 losses, counts and gradient.

Bounds, with u = 2^-24, R the largest |logit| of a live row: expf is within
2 ulp, l - top rounds by u R, so p is off by at most (4 R + 16) u relative, lse
by (4 R + 16) u absolute, sum f p likewise with 8 more roundings.  With
C = (8 R + 48) u (twice that sum) an entry of dlogits is off by at most
  C p (a E / N (|f - f.p| + 1) + 2 b / N (|lse| + 1)),
and the losses by C relative to the mean of their terms' magnitudes (sums run
over at most 4 + 5 + 8 fp32 additions before they are taken in double, below
the slack).  Counts are exact.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_layer_07_b200 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _inputs(T, seed, spread=1.5):
    r = np.random.default_rng(seed)
    lg = r.normal(0, spread, (T, 8)).astype(np.float32)
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :2].astype(np.int32)
    return r, lg, idx


def _call(lg, idx, mask=None, off=None, a=0.01, b=0.001, **kw):
    cfg = moe.Config(lg.shape[0], 256, 256)
    dev = lambda v, dt=None: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    off_t = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    return moe.balance_loss(cfg, dev(lg), dev(idx), token_mask=dev(mask), seq_offsets=off_t, balance_coef=a, z_coef=b, **kw)


def _check(lg, idx, mask=None, off=None, a=0.01, b=0.001):
    T = lg.shape[0]
    got = _call(lg, idx, mask, off, a, b)
    loss, counts, dl = oracle.balance_loss(lg, idx, mask, off, a, b)
    np.testing.assert_array_equal(got["counts"].cpu().numpy(), counts)
    live = np.zeros(T, bool)
    bounds = [0, T] if off is None else off
    live[bounds[0]:bounds[-1]] = True
    if mask is not None:
        live &= mask.astype(bool)
    n = max(1, int(live.sum()))
    g = got["dlogits"].cpu().numpy().astype(np.float64)
    assert np.all(g[~live] == 0)
    if live.any():
        l64 = lg[live].astype(np.float64)
        fin = np.where(np.isfinite(l64), l64, 0)
        C = (8 * np.abs(fin).max() + 48) * U
        top = l64.max(1, keepdims=True)
        ex = np.exp(l64 - top)
        p, lse = ex / ex.sum(1, keepdims=True), top + np.log(ex.sum(1, keepdims=True))
        lim = C * p * (a * 8 / n * 2 + 2 * b / n * (np.abs(lse) + 1)) + 1e-37
        assert np.all(np.abs(g[live] - dl[live]) <= lim)
        lz = float(np.mean(lse ** 2 + 1))
        got_loss = got["loss"].cpu().numpy().astype(np.float64)
        for i, mag in ((1, 8.0), (2, lz), (0, a * 8.0 + b * lz)):
            assert abs(got_loss[i] - loss[i]) <= 2 * C * mag
    else:
        assert not got["loss"].cpu().numpy().any()
    assert moe.get_device_error() == 0
    return got


@pytest.mark.parametrize("T", [1, 2, 31, 257, 1023, 1024, 1025, 5000, 20000])
def test_one_sequence(T):
    _, lg, idx = _inputs(T, T)
    _check(lg, idx)


@pytest.mark.parametrize("T,S", [(40, 3), (1024, 64), (3000, 7), (5000, 1500), (100, 5000), (17000, 33)])
def test_ragged_sequences_with_masks(T, S):
    r, lg, idx = _inputs(T, 11 * T + S)
    off = sorted(int(v) for v in r.integers(0, T + 1, S + 1))
    mask = (r.random(T) < 0.7).astype(np.uint8)
    if S > 3:
        mask[off[2]:off[3]] = 0  # a sequence without a live token
    _check(lg, idx, mask, off)
    _check(lg, idx, mask.astype(bool), None)


def test_many_sequences_in_one_chunk():
    # more sequences than are held at once: 1000 of one token, then 3000 empty ones, then the rest
    _, lg, idx = _inputs(2500, 5)
    off = list(range(1000)) + [1000] * 3000 + [1700, 1700, 2500]
    _check(lg, idx, None, off)


def test_masked_rows_are_not_read():
    r, lg, idx = _inputs(1500, 9)
    mask = (r.random(1500) < 0.5).astype(np.uint8)
    want = _call(lg, idx, mask)
    lg[mask == 0] = np.nan
    lg[np.flatnonzero(mask == 0)[::2]] = np.inf
    idx[mask == 0] = 1 << 30
    got = _call(lg, idx, mask)
    for k in ("loss", "counts", "dlogits"):
        assert torch.equal(want[k], got[k]), k
    assert moe.get_device_error() == 0
    none = _check(lg, np.zeros_like(idx), np.zeros(1500, np.uint8), [0, 700, 1500])
    assert not none["dlogits"].any() and not none["counts"].any()


def test_infinite_and_extreme_logits():
    _, lg, idx = _inputs(300, 2)
    lg[5, 3:] = -np.inf       # five experts of probability 0
    lg[7] = [3e38, -3e38, 0, 0, 0, 0, 0, 0]
    lg[7] = np.clip(lg[7], -1e4, 1e4)
    lg[9] = 0
    idx[5], idx[7], idx[9] = (0, 1), (0, 2), (0, 1)
    _check(lg, idx)
    lg[11, 2] = np.nan
    got = _call(lg, idx)
    assert torch.isnan(got["loss"]).all() and torch.isnan(got["dlogits"][11]).all()
    rest = torch.ones(300, dtype=torch.bool)
    rest[11] = False
    assert torch.isfinite(got["dlogits"][rest.cuda()]).all()


def test_a_loss_without_weight_does_not_spoil_the_sum():
    _, lg, idx = _inputs(50, 3)
    lg[4] = 1e20  # lse^2 passes fp32
    idx[4] = (0, 1)
    got = _call(lg, idx, b=0.0)
    assert torch.isinf(got["loss"][2]) and torch.isfinite(got["loss"][:2]).all() and torch.isfinite(got["dlogits"]).all()


def test_same_expert_twice_counts_twice():
    _, lg, idx = _inputs(70, 4)
    idx[:, 1] = idx[:, 0]
    _check(lg, idx)


def test_bad_index_is_flagged_and_not_counted():
    _, lg, idx = _inputs(70, 4)
    want = _call(lg, idx)["counts"].sum().item()
    idx[3, 1], idx[4, 0] = 8, -1
    got = _call(lg, idx)["counts"].sum().item()
    assert want == 140 and got == 138
    assert moe.get_device_error() == moe.DEVERR["EXPERT_INDEX"]


def test_bad_offsets_are_flagged():
    _, lg, idx = _inputs(2000, 4)
    for off in ([0, 900, 800, 2000], [-5, 2000], [0, 100, 2001]):
        _call(lg, idx, None, off)
        assert moe.get_device_error() == moe.DEVERR["OFFSETS"]


def test_no_tokens():
    got = _call(np.zeros((0, 8), np.float32), np.zeros((0, 2), np.int32), off=[0, 0, 0])
    assert not got["loss"].any() and got["counts"].shape == (2, 8) and not got["counts"].any()


def test_loss_without_gradient_and_given_outputs():
    _, lg, idx = _inputs(900, 6)
    want = _call(lg, idx)
    out = {"loss": torch.full((3,), 7.0, device="cuda"), "counts": torch.full((1, 8), 7, dtype=torch.int32, device="cuda")}
    got = _call(lg, idx, want_grad=False, out=out)
    assert got["dlogits"] is None and got["loss"] is out["loss"]
    assert torch.equal(got["loss"], want["loss"]) and torch.equal(got["counts"], want["counts"])


@pytest.mark.parametrize("T", [300, 9000, 40000])
def test_replays_from_a_graph_on_another_stream(T):
    r, lg, idx = _inputs(T, 8)
    off = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    cfg = moe.Config(T, 256, 256)
    lt, it = torch.from_numpy(lg).cuda(), torch.from_numpy(idx).cuda()
    ws = torch.full((moe.balance_loss_workspace_size(cfg, 2),), 255, dtype=torch.uint8, device="cuda")
    out = {"loss": torch.zeros(3, device="cuda"), "counts": torch.zeros((2, 8), dtype=torch.int32, device="cuda"),
           "dlogits": torch.zeros((T, 8), device="cuda")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.balance_loss(cfg, lt, it, seq_offsets=off, out=out, ws=ws)
    for seed in (1, 2):
        _, lg2, idx2 = _inputs(T, seed)
        lt.copy_(torch.from_numpy(lg2))
        it.copy_(torch.from_numpy(idx2))
        if ws.numel():
            ws.random_()  # nothing of the last call is needed
        graph.replay()
        want = moe.balance_loss(cfg, lt, it, seq_offsets=off)
        for k in want:
            assert torch.equal(out[k], want[k]), k
