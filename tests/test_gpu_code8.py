"""The 8-bit codes of pre-activations that are known exactly: a token with one value 1 has a row of W as its G and U.

The scale is exact.  The kernel rounds v (1 / s), 1 / s in fp32: off by 2^-24 of v / s, which is at most
127 (1 + 2^-8) < 127.5, so |v / s - c| <= 1/2 + 2^-17, and c is the nearest integer everywhere else.  (Half a step
alone does not hold: 129 2^-15 under the scale 129 2^-14 is a tie, whose product may come out above 1/2.)
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_layer_07_b200 as moe

pytestmark = pytest.mark.gpu


def test_codes_of_known_values():
    T = d = 256
    f = 512
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    cfg = moe.Config(T, d, f, capacity_factor=4.0)
    x = torch.eye(T, device="cuda", dtype=torch.bfloat16)
    w = [(rand(8, d, f) * 2.0 ** torch.randint(-40, 40, (8, d, f // 32, 1), generator=gen, device="cuda")
          .expand(8, d, f // 32, 32).reshape(8, d, f)).bfloat16() for _ in range(2)]
    # blocks full of ties: largest value 127.5 s with s = 129 2^-14 or 2^-3, the others odd multiples of s / 2
    half = torch.arange(32, device="cuda") * 2 - 31
    for i, step in enumerate((129 * 2.0 ** -15, 2.0 ** -4, 133 * 2.0 ** -12, 255 * 2.0 ** -9)):
        tie = (half * step).bfloat16()
        tie[31] = (254 * step)
        w[0][:, i::8, :32] = tie
        w[1][:, i::8, 32:64] = -tie
    w[0][:, 5, :32] = 0
    wd = torch.zeros((8, f, d), dtype=torch.bfloat16, device="cuda")
    wr = rand(8, d).bfloat16()
    ck = torch.full((moe.checkpoint_size_c8(cfg),), 255, dtype=torch.uint8, device="cuda")
    ws = torch.full((moe.workspace_size_train_c8(cfg),), 255, dtype=torch.uint8, device="cuda")
    moe.layer_forward_train_c8(cfg, x, wr, w[0], w[1], wd, ck, ws)
    kept = moe.checkpoint_views_c8(cfg, ck)
    route, perm = kept["route"].tolist(), kept["perm"].long()
    off = route[16:]
    assert off[8] == 2 * T
    for i, q in enumerate(("g", "u")):
        v = torch.cat([w[i][e][perm[off[e]:off[e + 1]]] for e in range(8)]).double().cpu().numpy()
        want, s = oracle.code8(v)
        codes, scale = kept[q + "_codes"].cpu().numpy().astype(np.int64), kept[q + "_scale"].double().cpu().numpy()
        assert np.array_equal(scale, s)
        step = np.repeat(s, 32, axis=1)
        ratio = np.divide(v, step, out=np.zeros_like(v), where=step > 0)
        assert np.all(np.abs(ratio - codes) <= 0.5 + 2.0 ** -17)
        clear = np.abs(np.abs(ratio - np.floor(ratio)) - 0.5) > 2.0 ** -17
        assert np.array_equal(codes[clear], want[clear]) and not clear.all()
        assert np.all(np.abs(oracle.decode8(codes, s) - v) <= step / 2 * (1 + 2.0 ** -16))
    assert moe.get_device_error() == 0
