"""Weight gradients of the last tokens of a long batch: their rows lie past 2^32 codes and values.

dout is zero for all tokens but the last n, so dG, dU and the products with dout are exactly zero for the others and
only the last rows are in the sums.  A row's dG, dU and w H do not depend on the batch, so against the batch of the
last n tokens alone an entry differs by the order of its sum of n_e rows on either side, (n_e + 2) 2^-23 of the terms'
magnitudes, and by one rounding to bf16 on either side, 2^-8 of it.  The magnitudes are formed here from the decoded
pre-activations in fp32 (off by far less than the 2% that are added).
"""
from __future__ import annotations

import pytest
import torch

import sparse_moe_layer_07_b200 as moe

pytestmark = pytest.mark.gpu


def test_weight_gradients_past_32_bits():
    T, n, d, f = 70000, 600, 256, 32768
    gen = torch.Generator(device="cuda").manual_seed(17)

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(std=std, generator=gen)

    x, dout = normal(T, d), normal(T, d)
    dout[:T - n] = 0
    wr, wg, wu, wd = (normal(8, d, std=d ** -0.5), normal(8, d, f, std=d ** -0.5), normal(8, d, f, std=d ** -0.5),
                      normal(8, f, d, std=f ** -0.5))

    def step(lo):
        c = moe.Config(T - lo, d, f, capacity_factor=4.0)
        ck = torch.empty(moe.checkpoint_size_c8(c), dtype=torch.uint8, device="cuda")
        ws = torch.empty(moe.workspace_size_train_c8(c), dtype=torch.uint8, device="cuda")
        moe.layer_forward_train_c8(c, x[lo:], wr, wg, wu, wd, ck, ws)
        return moe.layer_backward_c8(c, x[lo:], wr, wg, wu, wd, dout[lo:], ck, ws), moe.checkpoint_views_c8(c, ck)

    got, _ = step(0)
    want, kept = step(T - n)
    assert not got["dx"][:T - n].any() and torch.equal(got["dx"][T - n:], want["dx"])
    off = kept["route"][16:].tolist()
    assert off[8] == 2 * n
    for e in range(8):
        r = slice(off[e], off[e + 1])
        tok = kept["perm"][r].long()
        g, u = ((kept[q + "_codes"][r].float().view(-1, f // 32, 32) * kept[q + "_scale"][r].float()[:, :, None]).view(-1, f)
                for q in ("g", "u"))
        a, go, w = x[T - n:][tok].float().abs(), dout[T - n:][tok].float(), kept["row_scale"][r][:, None]
        dhu, sig = w * (go @ wd[e].float().t()), torch.sigmoid(g)
        terms = {"dw_gate": (a, (dhu * u * sig * (1 + g * (1 - sig))).abs()), "dw_up": (a, (dhu * g * sig).abs()),
                 "dw_down": ((w * g * sig * u).abs(), go.abs())}
        t = (off[e + 1] - off[e] + 2) * 2.0 ** -23
        for q, (rows, cols) in terms.items():
            p, s = got[q][e].float(), want[q][e].float()
            lim = 2 * t * 1.02 * (rows.t() @ cols) + 2.0 ** -8 * (p.abs() + s.abs())
            assert s.any() and ((p - s).abs() <= lim).all(), (q, e)
    assert moe.get_device_error() == 0
