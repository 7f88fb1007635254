"""moe_balance_loss on large batches: blocks that take several chunks of 1024 tokens (more than three chunks an SM),
chunks of padding behind live ones, chunks that meet more sequences than are held at once, and searches of more
than 4096 sequences.

Bounds, with u = 2^-24 and R the largest |logit| of a live row: l - top rounds by 2 R u; __expf is within
2 + 1.173 |x| ulp of 2 u each, so e^(l - top) is off by (6.7 R + 4) u relative, their sum by 7 u more, the quotient
by 5 u more: p by at most (13.4 R + 20) u.  lse is off by (6.7 R + 11) u from the sum, 12 u from __logf and its own
rounding R u + 3 u.  f = counts / (2 n) has two roundings, sum f p eight more.  C = (16 R + 64) u covers each, so an
entry of dlogits is off by at most
  C p (a E / N (|f - f.p| + 1) + 2 b / N (|lse| + 1)).
A chunk's sums take 1 + 5 + 16 fp32 additions, within C, and are added in double.  The losses are off by at most
2 C times the mean of their terms' magnitudes (8 for balance, lse^2 + 1 for z).  Counts are exact.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_layer_07_b200 as moe

U = 2.0 ** -24
A, B = 0.01, 0.001


def _formula(lg, idx, mask, off, a, b):
    """The losses, counts and gradient in 64 bits over whole arrays, and what the bounds take: live, p, lse."""
    T, S = lg.shape[0], len(off) - 1
    off = np.asarray(off, dtype=np.int64)
    t = np.arange(T)
    live = (t >= off[0]) & (t < off[-1])
    if mask is not None:
        live &= mask.astype(bool)
    seq = np.searchsorted(off, t, side="right") - 1  # the last sequence that begins at or before t, empty ones passed
    seq = np.where(live, seq, 0)
    keys = (seq[:, None] * 8 + idx)[live]
    counts = np.bincount(keys.reshape(-1), minlength=S * 8).reshape(S, 8)
    n = int(live.sum())
    per = np.maximum(np.bincount(seq[live], minlength=S), 1)
    f = (counts / (2.0 * per[:, None]))[seq]
    l64 = lg.astype(np.float64)
    top = l64.max(1, keepdims=True)
    ex = np.exp(l64 - top)
    p = ex / ex.sum(1, keepdims=True)
    lse = top[:, 0] + np.log(ex.sum(1))
    fp = (f * p).sum(1)
    m = max(n, 1)
    balance, z = 8.0 * fp[live].sum() / m, (lse[live] ** 2).sum() / m
    dl = p * (a * 8.0 / m * (f - fp[:, None]) + 2.0 * b / m * lse[:, None])
    dl[~live] = 0
    return np.array([a * balance + b * z, balance, z]), counts, dl, live, p, lse


def _inputs(T, seed):
    r = np.random.default_rng(seed)
    lg = r.normal(0, 1.5, (T, 8)).astype(np.float32)
    top = np.argpartition(-lg, 1, axis=1)[:, :2]
    return r, lg, top.astype(np.int32)


def _cuts(r, lo, hi, n_seq):
    """n_seq + 1 offsets from lo to hi."""
    return [lo, *sorted(int(v) for v in r.integers(lo, hi + 1, n_seq - 1)), hi]


def test_formula_is_the_oracles():
    r, lg, idx = _inputs(200, 1)
    for S, mask in ((1, None), (7, r.random(200) < 0.7), (300, r.random(200) < 0.7)):
        off = _cuts(r, 3, 190, S)
        loss, counts, dl, live, _, _ = _formula(lg, idx, mask, off, A, B)
        want = oracle.balance_loss(lg, idx, mask, off, A, B)
        assert np.allclose(loss, want[0], rtol=1e-12) and np.array_equal(counts, want[1])
        assert np.allclose(dl, want[2], rtol=1e-10, atol=1e-18) and not dl[~live].any()


def _check(lg, idx, mask, off, repeats=1):
    T = lg.shape[0]
    cfg = moe.Config(T, 256, 256)
    dev = [None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda()
           for v in (lg, idx, mask, np.asarray(off, dtype=np.int32))]
    ws = torch.full((moe.balance_loss_workspace_size(cfg, len(off) - 1),), 255, dtype=torch.uint8, device="cuda")
    call = lambda: moe.balance_loss(cfg, dev[0], dev[1], token_mask=dev[2], seq_offsets=dev[3], balance_coef=A,  # noqa: E731
                                    z_coef=B, ws=ws)
    got = call()
    loss, counts, dl, live, p, lse = _formula(lg, idx, mask, off, A, B)
    np.testing.assert_array_equal(got["counts"].cpu().numpy(), counts)
    n = max(1, int(live.sum()))
    C = (16 * (np.abs(lg[live]).max() if live.any() else 0.0) + 64) * U
    g = got["dlogits"].cpu().numpy().astype(np.float64)
    assert not g[~live].any()
    lim = C * p * (A * 8 / n * 2 + 2 * B / n * (np.abs(lse)[:, None] + 1)) + 1e-37
    assert np.all(np.abs(g - dl)[live] <= lim[live])
    lz = float(np.mean(lse[live] ** 2 + 1)) if live.any() else 0.0
    out = got["loss"].cpu().numpy().astype(np.float64)
    for i, mag in ((1, 8.0), (2, lz), (0, A * 8.0 + B * lz)):
        assert abs(out[i] - loss[i]) <= 2 * C * mag, (i, out[i], loss[i])
    for _ in range(repeats):
        again = call()
        for k in got:
            assert torch.equal(again[k], got[k]), k
    assert moe.get_device_error() == 0


# live tokens end at `end`: a few chunks of padding, one that ends inside a chunk, most chunks (on 148 SMs blocks take
# a second chunk from token 454656 on and a third from 909312)
@pytest.mark.gpu
@pytest.mark.parametrize("T,end,S,masked", [
    (500000, 499000, 60, True), (500000, 455000, 1, False), (600000, 460000, 40, True), (1 << 20, 1027605, 1000, True),
    (1 << 20, 300000, 200, False), (1 << 20, 1 << 20, 1, True), (1000001, 5, 2, False)])
def test_blocks_of_several_chunks_with_padding(T, end, S, masked):
    r, lg, idx = _inputs(T, T + S)
    _check(lg, idx, r.random(T) < 0.9 if masked else None, _cuts(r, 0, end, S), repeats=20)


@pytest.mark.gpu
@pytest.mark.parametrize("T,S", [(5000, 9000), (16384, 4097), (20000, 6000), (500000, 100000), (600000, 1300000)])
def test_many_sequences(T, S):
    """More than 4096 sequences, and at two a token more of them in a chunk than are held at once."""
    r, lg, idx = _inputs(T, T + S)
    _check(lg, idx, r.random(T) < 0.8, _cuts(r, T // 100, T - T // 50, S), repeats=3)


@pytest.mark.gpu
def test_runs_of_empty_sequences_inside_a_chunk():
    for T in (5000, 20000, 500000):
        r, lg, idx = _inputs(T, T)
        t = T - 2500
        off = [*range(t - 900, t), *[t] * 3500, *[t + 700] * 1500, t + 701, T]
        _check(lg, idx, None, off, repeats=3)
        _check(lg, idx, r.random(T) < 0.5, off)
