"""Microscaled 4-bit experts against the oracle.

quantise / dequantise: every decision is exact in fp32 (scales are powers of
two), so codes, scales and decoded weights are compared bit for bit.

Products: operands are exact, so with t(n) = (n + 2) 2^-23 (n products added in
fp32, truncation allowed)
  g, u   off by at most e = t(d) sum |x^| |w^|;
  h      by |silu'| |u| e_g + |silu(g)| e_u + 2^-20 |silu(g) u| + e_g e_u, with
         |silu'| <= 1.1: E_h;
  h^     by E_h + 2^-4 (|h| + E_h) + 2^-10 2^x (half a step of a normal and of a
         subnormal e4m3 number), its scale 2^x such that the block's largest
         element lies in (224, 448] of it, up to E_h;
  y      at the GPU's own h^, by |w| t(f) sum |h^| |d^|.
The layer's output is the combine of y bit for bit.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_layer_07_b200 as moe
from synth import configs, normal

from parity_util import LayerInputs, to_dev

pytestmark = pytest.mark.gpu

W = configs.WORKLOADS


def _bits(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def _as_np(t):
    return t.cpu().view(torch.uint16).numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def _weights(K, N, seed, hard):
    r = np.random.default_rng(seed)
    w = r.normal(0, 1, (8, K, N))
    if hard:
        w *= 2.0 ** r.integers(-60, 60, (8, K // 32, 1, N)).repeat(32, 2).reshape(8, K, N)
        w[0, :32] = r.integers(-28, 29, (32, N)) * 0.25  # ties on every midpoint
        w[1, :32] = 0
        w[1, 5, ::2] = -0.0
        w[2, :32] *= 2.0 ** -20 * 1e-36  # subnormal in bf16
        w[3, :32] = 3.3e38 * r.choice([-1, 0.3, 0.9, 1], (32, N))
        w[4, 7, 3], w[4, 40, 5], w[4, 41, 6] = np.nan, np.inf, -np.inf
        w[5, :32] = 1.75 * 2.0 ** r.integers(-8, 8, (1, N))
        w[5, 3, ::3] *= 1.004  # one bf16 step over 1.75
    return _bits(w)


@pytest.mark.parametrize("K,N,hard", [(128, 128, True), (384, 256, True), (256, 640, False), (1536, 128, False)])
def test_quantise_and_dequantise_are_exact(K, N, hard):
    w = _weights(K, N, K + N, hard)
    cfg = moe.Config(0, 256, 256)
    codes, scales = moe.quantize_mx4(cfg, w.cuda())
    back = moe.dequantize_mx4(cfg, codes, scales)
    bits = _as_np(w)
    for e in range(8):
        c, x = oracle.mx4_blocks(bits[e])
        want_c, want_s = oracle.mx4_pack(c, x)
        assert np.array_equal(codes[e].cpu().numpy(), want_c), e
        assert np.array_equal(scales[e].cpu().numpy(), want_s), e
        v = oracle.mx4_values(c, x)
        got = back[e].float().cpu().numpy().astype(np.float64)
        assert np.array_equal(got, v, equal_nan=True) and np.array_equal(np.signbit(got[~np.isnan(v)]), np.signbit(v[~np.isnan(v)])), e


CASES = {
    "one_token": dict(T=1, d=256, f=128, capacity_factor=4.0),
    "few": dict(T=7, d=512, f=384, capacity_factor=4.0),
    "decode": dict(T=32, d=256, f=1024, capacity_factor=4.0),
    "decode_two": dict(T=60, d=256, f=256, capacity_factor=4.0, logit_bias=(60.0, 50.0, 0, 0, 0, 0, 0, 0)),
    "decode_skew": dict(T=230, d=256, f=256, capacity_factor=4.0, logit_bias=(60.0, 50.0, 0, 0, 0, 0, 0, 0)),
    "tiles_of_32": dict(T=96, d=256, f=384, capacity_factor=4.0),
    "tiles_of_64": dict(T=130, d=512, f=256, capacity_factor=4.0),
    # 190 rows on each of two experts: three tiles of 64, the last at the middle of a 128-row block of scales
    "tiles_of_64_skew": dict(T=190, d=256, f=256, capacity_factor=4.0, logit_bias=(60.0, 50.0, 0, 0, 0, 0, 0, 0)),
    "last_streaming": dict(T=256, d=256, f=640, capacity_factor=1.25),
    "first_tiled": dict(T=257, d=256, f=256, capacity_factor=4.0),
    "ragged": dict(T=700, d=512, f=384, capacity_factor=1.25),
    "full_tiles": dict(T=512, d=256, f=256, capacity_factor=4.0, logit_bias=(60.0, 50.0, 0, 0, 0, 0, 0, 0)),
    "wide": dict(T=300, d=1536, f=256, capacity_factor=4.0),
    # the layer's down tiles have 128 columns up to here, then 192, then 256
    "columns_192": dict(T=600, d=1536, f=256, capacity_factor=4.0),
    "columns_256": dict(T=8192, d=256, f=128, capacity_factor=4.0),
    "long": dict(T=40, d=256, f=8192, capacity_factor=4.0),
}


@pytest.fixture(scope="module", params=sorted(CASES))
def ffn(request):
    w = configs.scaled(W["mid_bf16"], name=f"mx_{request.param}", **CASES[request.param])
    L = LayerInputs(w)
    c, D = L.cfg, L.dev
    qw = moe.MxExperts(c, D["wg"], D["wu"], D["wd"])
    idx, wts, _ = moe.router_topk(c, D["x"], D["wr"], D["bias"])
    disp = moe.dispatch(c, D["x"], idx, wts)
    # 255 is a NaN code and a NaN scale: rows that do not exist may not reach results
    ws = torch.full((moe.expert_ffn_mx4_workspace_size(c),), 255, dtype=torch.uint8, device="cuda")
    n = int(disp["offsets"][8])
    disp["x_perm"][n:] = float("nan")
    y = torch.full((2 * w.T, w.d), 7.0, device="cuda")
    moe.expert_ffn_mx4(c, disp["x_perm"], disp["offsets"], qw, disp["row_scale"], y=y, ws=ws)
    torch.cuda.synchronize()
    assert moe.get_device_error() == 0
    return w, L, qw, idx, wts, disp, ws, y, n


def _decoded(codes, scales, off):
    """Values and exponents of the rows below off[8], from codes and scale blocks."""
    n, K = int(off[8]), codes.shape[1]
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    x = np.zeros((n, K // 32), dtype=np.int64)
    tile = 0
    k = np.arange(K // 32)
    for e in range(8):
        for r in range(int(off[e]), int(off[e + 1])):
            i = r - int(off[e])
            x[r] = scales[tile + i // 128, k // 4, i % 32 * 16 + i % 128 // 32 * 4 + k % 4].astype(np.int64) - 127
        tile += -(-int(off[e + 1] - off[e]) // 128)
    return oracle.e4m3_values(codes[:n]) * np.ldexp(1.0, np.repeat(x, 32, axis=1)), x


def test_rows_of_x_are_coded_exactly(ffn):
    w, L, qw, idx, wts, disp, ws, y, n = ffn
    off = disp["offsets"].cpu().numpy()
    v = moe.mx4_workspace_views(L.cfg, ws)
    got, x = _decoded(v["x_codes"], v["x_scales"], off)
    want, wx = oracle.mx8_rows(oracle.to_f64(L.x)[disp["perm"].cpu().numpy()[:n]])
    assert np.array_equal(got, want) and np.array_equal(x, wx)


def test_products_within_their_bounds(ffn):
    w, L, qw, idx, wts, disp, ws, y, n = ffn
    off = disp["offsets"].cpu().numpy()
    v = moe.mx4_workspace_views(L.cfg, ws)
    xh, _ = _decoded(v["x_codes"], v["x_scales"], off)
    hh, hx = _decoded(v["h_codes"], v["h_scales"], off)
    got = y.cpu().numpy().astype(np.float64)
    assert np.all(got[n:] == 7.0)  # rows behind the last one stay as they were
    scale = disp["row_scale"].cpu().numpy().astype(np.float64)
    t = lambda k: (k + 2) * 2.0 ** -23  # noqa: E731
    for e in range(8):
        r = slice(int(off[e]), int(off[e + 1]))
        if r.start == r.stop:
            continue
        wg, wu, wd = (oracle.mx4_values(*oracle.mx4_blocks(q[e])) for q in (L.wg, L.wu, L.wd))
        a, h8 = xh[r], hh[r]
        g, u = a @ wg, a @ wu
        eg, eu = t(w.d) * (np.abs(a) @ np.abs(wg)), t(w.d) * (np.abs(a) @ np.abs(wu))
        sl = oracle.silu(g)
        h = sl * u
        eh = 1.1 * np.abs(u) * eg + np.abs(sl) * eu + 2.0 ** -20 * np.abs(h) + 1.1 * eg * eu
        unit = np.ldexp(1.0, np.repeat(hx[r], 32, axis=1))
        assert np.all(np.abs(h8 - h) <= eh + 2.0 ** -4 * (np.abs(h) + eh) + 2.0 ** -10 * unit), e
        top = np.abs(h).reshape(h.shape[0], -1, 32).max(2) / np.ldexp(1.0, hx[r])
        slack = eh.reshape(h.shape[0], -1, 32).max(2) / np.ldexp(1.0, hx[r])
        assert np.all(top <= 448 + slack) and np.all((top > 224 - slack) | (hx[r] == -127)), e
        want = scale[r][:, None] * (h8 @ wd)
        lim = scale[r][:, None] * t(w.f) * (np.abs(h8) @ np.abs(wd)) + 1e-37
        assert np.all(np.abs(got[r] - want) <= lim), (e, float(np.max(np.abs(got[r] - want) / lim)))


def test_layer_is_the_combine_of_the_experts(ffn):
    w, L, qw, idx, wts, disp, ws, y, n = ffn
    c, D = L.cfg, L.dev
    big = torch.full((moe.workspace_size_mx4(c),), 255, dtype=torch.uint8, device="cuda")
    stats = torch.zeros(26, dtype=torch.int32, device="cuda")
    out = moe.layer_forward_mx4(c, D["x"], D["wr"], qw, logit_bias=D["bias"], ws=big, stats=stats)
    want = moe.combine(c, y, disp["slot_of"], wts)
    assert torch.equal(out, want)
    assert torch.equal(stats[:8], disp["counts_raw"]) and int(stats[25]) == 2 * w.T - n
    again = moe.layer_forward_mx4(c, D["x"], D["wr"], moe.MxExperts.from_codes(*qw.tensors()), logit_bias=D["bias"])
    assert torch.equal(out, again)
    assert moe.get_device_error() == 0


def test_without_row_scale(ffn):
    w, L, qw, idx, wts, disp, ws, y, n = ffn
    plain = moe.expert_ffn_mx4(L.cfg, disp["x_perm"], disp["offsets"], qw)
    scaled = disp["row_scale"][:n, None] * plain[:n]
    # one rounding of a product on either side (of partial sums where K is split: one for each)
    parts = 8 if 2 * w.T <= 512 else 1
    assert torch.all((scaled - y[:n]).abs() <= parts * 2.0 ** -23 * plain[:n].abs().max())


def test_near_the_bf16_layer():
    """The whole quantised layer stays within what the formats lose: 4-bit weights and 8-bit rows, each taken as
    independent errors of the root mean square stated with the formats (11% and 3%), on three products."""
    w = configs.scaled(W["mid_bf16"], name="mx_near", T=600, d=512, f=1024, capacity_factor=4.0)
    L = LayerInputs(w)
    D = L.dev
    full = moe.layer_forward(L.cfg, D["x"], D["wr"], D["wg"], D["wu"], D["wd"]).float()
    got = moe.layer_forward_mx4(L.cfg, D["x"], D["wr"], moe.MxExperts(L.cfg, D["wg"], D["wu"], D["wd"])).float()
    rel = float((got - full).norm() / full.norm())
    # gate, up and down each add one weight and one row error: sqrt(3 (0.12^2 + 0.03^2)) = 0.214; silu' up to 1.1 on gate
    assert rel <= 0.24, rel
    # the same layer on the dequantised weights differs by the rows' 8 bits alone
    deq = [moe.dequantize_mx4(L.cfg, *moe.quantize_mx4(L.cfg, D[k])) for k in ("wg", "wu", "wd")]
    mid = moe.layer_forward(L.cfg, D["x"], D["wr"], *deq).float()
    assert float((got - mid).norm() / mid.norm()) <= 0.06


def test_nan_rows_and_blocks_stay_where_they_are():
    w = configs.scaled(W["mid_bf16"], name="mx_nan", T=300, d=256, f=256, capacity_factor=4.0)
    L = LayerInputs(w)
    D = L.dev
    wg = D["wg"].clone()
    x = D["x"].clone()
    idx, wts, _ = moe.router_topk(L.cfg, x, D["wr"])
    disp = moe.dispatch(L.cfg, x, idx, wts)
    qw = moe.MxExperts(L.cfg, wg, D["wu"], D["wd"])
    base = moe.expert_ffn_mx4(L.cfg, disp["x_perm"], disp["offsets"], qw)
    xp = disp["x_perm"].clone()
    xp[5, 17], xp[9, 200] = float("inf"), float("nan")
    got = moe.expert_ffn_mx4(L.cfg, xp, disp["offsets"], qw)
    keep = torch.ones(600, dtype=torch.bool, device="cuda")
    keep[5] = keep[9] = False
    assert torch.isnan(got[5]).all() and torch.isnan(got[9]).all() and torch.equal(got[keep], base[keep])
    # a NaN in one expert's weights: that expert's rows, no other's
    wg[3, 40, 7] = float("nan")
    bad = moe.expert_ffn_mx4(L.cfg, disp["x_perm"], disp["offsets"], moe.MxExperts(L.cfg, wg, D["wu"], D["wd"]))
    off = disp["offsets"].cpu().tolist()
    mine = torch.zeros(600, dtype=torch.bool, device="cuda")
    mine[off[3]:off[4]] = True
    assert torch.isnan(bad[mine]).all() and torch.equal(bad[~mine], base[~mine])
    assert moe.get_device_error() == 0


def test_bad_offsets_and_indices_are_flagged():
    cfg = moe.Config(40, 256, 256, capacity_factor=4.0)
    qw = moe.MxExperts(cfg, *(torch.zeros((8, 256, 256), dtype=torch.bfloat16, device="cuda") for _ in range(3)))
    xp = torch.zeros((80, 256), dtype=torch.bfloat16, device="cuda")
    for off in ([0, 9, 5, 80, 80, 80, 80, 80, 80], [0, 10, 20, 30, 40, 50, 60, 70, 81], [-1, 0, 0, 0, 0, 0, 0, 0, 4]):
        moe.expert_ffn_mx4(cfg, xp, torch.tensor(off, dtype=torch.int32, device="cuda"), qw)
        assert moe.get_device_error() == moe.DEVERR["OFFSETS"], off


def test_no_tokens():
    cfg = moe.Config(0, 256, 256)
    z = torch.zeros((8, 256, 256), dtype=torch.bfloat16, device="cuda")
    qw = moe.MxExperts(cfg, z, z, z)
    out = moe.layer_forward_mx4(cfg, z[0, :0], torch.zeros((8, 256), dtype=torch.bfloat16, device="cuda"), qw)
    assert out.shape == (0, 256)


@pytest.mark.parametrize("T,cf", [(1, 4.0), (32, 4.0), (700, 1.25)])
def test_replays_from_a_graph(T, cf):
    w = configs.scaled(W["mid_bf16"], name=f"mx_graph_{T}", T=T, d=256, f=384, capacity_factor=cf)
    L = LayerInputs(w)
    D, c = L.dev, L.cfg
    qw = moe.MxExperts(c, D["wg"], D["wu"], D["wd"])
    x_in = D["x"].clone()
    ws = torch.full((moe.workspace_size_mx4(c),), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x_in)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.layer_forward_mx4(c, x_in, D["wr"], qw, out=out, ws=ws)
    for seed in (0, 7):
        x_in.copy_(to_dev(normal(3, 50 + seed, (T, 256), dtype="bf16")))
        graph.replay()
        want = moe.layer_forward_mx4(c, x_in, D["wr"], qw)
        assert torch.equal(out, want)
    assert moe.get_device_error() == 0


def test_offsets_past_32_bits():
    """140000 rows of 32768 columns of H, more than 2^32 codes: the last tokens' outputs are those of a batch of them."""
    T, n, d, f = 70000, 600, 256, 32768
    gen = torch.Generator(device="cuda").manual_seed(12)

    def normal_(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(std=std, generator=gen)

    x, wr = normal_(T, d), normal_(8, d, std=d ** -0.5)
    c = moe.Config(T, d, f, capacity_factor=4.0)
    qw = moe.MxExperts(c, normal_(8, d, f, std=d ** -0.5), normal_(8, d, f, std=d ** -0.5), normal_(8, f, d, std=f ** -0.5))
    out = moe.layer_forward_mx4(c, x, wr, qw)
    last = moe.layer_forward_mx4(moe.Config(n, d, f, capacity_factor=4.0), x[T - n:], wr, qw)
    assert torch.equal(out[T - n:], last)
    assert moe.get_device_error() == 0


def test_batches_on_several_streams_at_once():
    """One set of weights, a batch and a scratch for each stream: one token, decode, and both sizes of row tiles."""
    L = LayerInputs(configs.scaled(W["mid_bf16"], name="mx_streams", T=700, d=256, f=384, capacity_factor=4.0))
    D = L.dev
    qw = moe.MxExperts(L.cfg, D["wg"], D["wu"], D["wd"])
    jobs = []
    for T in (1, 32, 130, 700):
        c = moe.Config(T, 256, 384, capacity_factor=4.0)
        jobs.append((c, D["x"][:T].contiguous(), torch.empty(moe.workspace_size_mx4(c), dtype=torch.uint8, device="cuda")))
    want = [moe.layer_forward_mx4(c, x, D["wr"], qw, ws=ws) for c, x, ws in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [moe.layer_forward_mx4(c, x, D["wr"], qw, ws=ws, stream=st)
           for _ in range(5) for (c, x, ws), st in zip(jobs, streams)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert torch.equal(out, want[i % len(jobs)]), i
    assert moe.get_device_error() == 0


def test_trained_then_served():
    """The set in use: a training step with 8-bit checkpoints and the balance loss, an update, the result served in 4 bits."""
    w = configs.scaled(W["mid_bf16"], name="mx_serve", T=400, d=256, f=512, capacity_factor=1.25)
    L = LayerInputs(w)
    c, D = L.cfg, L.dev
    ws = {k: D[k].clone() for k in ("wr", "wg", "wu", "wd")}
    ck = torch.empty(moe.checkpoint_size_c8(c), dtype=torch.uint8, device="cuda")
    sc = torch.empty(moe.workspace_size_train_c8(c), dtype=torch.uint8, device="cuda")
    out = moe.layer_forward_train_c8(c, D["x"], *ws.values(), ck, sc)
    v = moe.checkpoint_views_c8(c, ck)
    aux = moe.balance_loss(c, v["logits"], v["topk_idx"], balance_coef=0.01, z_coef=0.001)
    g = moe.layer_backward_c8(c, D["x"], *ws.values(), out, ck, sc, dlogits=aux["dlogits"])
    for k, q in (("wr", "dw_router"), ("wg", "dw_gate"), ("wu", "dw_up"), ("wd", "dw_down")):
        assert torch.isfinite(g[q].float()).all() and g[q].any()
        ws[k] -= 1e-3 * g[q]
    served = moe.layer_forward_mx4(c, D["x"], ws["wr"], moe.MxExperts(c, ws["wg"], ws["wu"], ws["wd"]))
    exact = moe.layer_forward(c, D["x"], *ws.values())
    assert float((served.float() - exact.float()).norm() / exact.float().norm()) <= 0.24
    assert moe.get_device_error() == 0
