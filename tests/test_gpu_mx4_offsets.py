"""moe_expert_ffn_mx4 on a table whose first expert does not start at row 0: the rows in front of it are nobody's.
A row's result depends on its own values alone, so the same rows moved up by `first` give the same bits."""
from __future__ import annotations

import pytest
import torch

import sparse_moe_layer_07_b200 as moe

pytestmark = pytest.mark.gpu


# rows an expert, in tiles of 32, of 64 and of 128; ends inside a 32- and a 128-row block of scales
@pytest.mark.parametrize("T,counts", [
    (96, (40, 0, 1, 5, 0, 33, 0, 7)), (130, (70, 0, 1, 3, 0, 0, 20, 9)), (200, (3, 129, 0, 0, 0, 0, 0, 10)),
    (700, (300, 0, 129, 128, 1, 0, 200, 77))])
@pytest.mark.parametrize("first", [1, 100, 200])
def test_rows_in_front_of_the_first_expert(T, counts, first):
    d, f, rows = 512, 384, 2 * T
    n = sum(counts)
    first = min(first, rows - n)
    assert first > 0
    gen = torch.Generator(device="cuda").manual_seed(T + first)
    normal = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)  # noqa: E731
    cfg = moe.Config(T, d, f, capacity_factor=4.0)
    qw = moe.MxExperts(cfg, normal(8, d, f), normal(8, d, f), normal(8, f, d))
    off = torch.tensor([0, *counts], dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)
    x, scale = normal(n, d), normal(n).float()

    def run(at):
        # 255 is a NaN code and a NaN scale
        ws = torch.full((moe.expert_ffn_mx4_workspace_size(cfg),), 255, dtype=torch.uint8, device="cuda")
        xp = torch.full((rows, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        rs = torch.full((rows,), float("nan"), device="cuda")
        y = torch.full((rows, d), 7.0, device="cuda")
        xp[at:at + n], rs[at:at + n] = x, scale
        moe.expert_ffn_mx4(cfg, xp, off + at, qw, rs, y=y, ws=ws)
        assert (y[:at] == 7.0).all() and (y[at + n:] == 7.0).all()
        return y[at:at + n]

    want = run(0)
    assert torch.isfinite(want).all()
    assert torch.equal(run(first), want)
    assert moe.get_device_error() == 0
