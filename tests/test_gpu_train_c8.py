"""The training pair with 8-bit activation checkpoints against the oracle.

Checkpoint: the fp32 pre-activation of the tensor cores differs from the fp64
one by at most e = (d + 2) 2^-23 sum_k |x_k w_k| (each of d products added in
fp32, truncation allowed), so with the decoded scale s an element is off by at
most e + s / 2 (1 + 2^-6): half a step, and the step's own rounding moves the
quotient by less than 2^-7 of itself times one.

Gradients: the oracle differentiates at the GPU's own decoded G, U with its
routing, in fp64, so what is left is arithmetic.  With b = 2^-8 (a rounding to
bf16, half a step) and t(n) = (n + 2) 2^-23 (a sum of n fp32 terms), relative
to the same products of absolute values:
  dHu       t(d)                                     E_h  = t(d) |dout| |Wd|^T
  dG        b + 2^-16 (expf, sigmoid), and E_h       E_g  = w |u| s' E_h + (b + 2^-16) |dG|
  dU        likewise with |silu(g)|
  dW_gate   E_g through |X|^T, t(rows), b on the result; dW_up, dW_down alike
  dx        E_g |Wg|^T + E_u |Wu|^T, t(2 f), the router's part, b
  dweight   E_h |h| + (t(f) + 2^-16) |dHu h|; dlogits w (its error + its mean's) + 2^-20
  dw_router, dbias: that through |x|, t(T), b.
s' is bounded by sig (1 + |g| (1 - sig)).  Every entry is held to its own bound.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_layer_07_b200 as moe
from synth import configs, normal

from parity_util import LayerInputs, to_dev, to_np64

pytestmark = pytest.mark.gpu

W = configs.WORKLOADS
KEYS = ("dx", "dw_router", "dbias", "dw_gate", "dw_up", "dw_down")
CASES = {
    "ragged": dict(T=700, d=256, f=512, capacity_factor=1.25),
    "drop": dict(T=513, d=512, f=256, capacity_factor=0.5),
    "one_token": dict(T=1, d=256, f=256, capacity_factor=4.0),
    "few_rows": dict(T=40, d=256, f=768, capacity_factor=4.0),
    # experts 2..7 have no rows
    "two_experts": dict(T=272, d=256, f=256, capacity_factor=4.0, logit_bias=(60.0, 50.0, 0, 0, 0, 0, 0, 0)),
    "wide": dict(T=130, d=1536, f=512, capacity_factor=4.0),
    # d of 2048 and more: the dH kernel's other split of its epilogue
    "wider": dict(T=300, d=2304, f=512, capacity_factor=1.25),
}


def _buffers(cfg, fill=None):
    ck = torch.empty(moe.checkpoint_size_c8(cfg), dtype=torch.uint8, device="cuda")
    ws = torch.empty(moe.workspace_size_train_c8(cfg), dtype=torch.uint8, device="cuda")
    if fill is not None:
        ck.fill_(fill)
        ws.fill_(fill)
    return ck, ws


class Step:
    def __init__(self, name, over=None):
        self.w = configs.scaled(W["mid_bf16"], name=f"c8_{name}", **dict(CASES[name], **(over or {})))
        self.L = L = LayerInputs(self.w)
        self.cfg, D = L.cfg, L.dev
        self.weights = (D["wr"], D["wg"], D["wu"], D["wd"])
        self.go = normal(configs.SEED, 907, (self.w.T, self.w.d), dtype="bf16")
        self.aux = normal(configs.SEED, 908, (self.w.T, 8), std=0.05, dtype="f32")
        # 255 bytes are NaN in bf16 and fp32: nothing that a call did not write may reach its results
        self.ck, self.ws = _buffers(self.cfg, 255)

    def forward(self):
        return moe.layer_forward_train_c8(self.cfg, self.L.dev["x"], *self.weights, self.ck, self.ws,
                                          logit_bias=self.L.dev["bias"])

    def backward(self, **kw):
        return moe.layer_backward_c8(self.cfg, self.L.dev["x"], *self.weights, to_dev(self.go), self.ck, self.ws, **kw)


@pytest.fixture(scope="module", params=sorted(CASES))
def step(request):
    s = Step(request.param)
    s.out = s.forward()
    s.ws.fill_(255)  # the backward needs nothing of the forward's scratch
    s.grads = s.backward(dlogits=torch.from_numpy(s.aux).cuda())
    torch.cuda.synchronize()
    v = moe.checkpoint_views_c8(s.cfg, s.ck)
    s.kept = {k: (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy() for k, t in v.items()}
    route = s.kept.pop("route")
    s.kept.update(counts_raw=route[:8], counts_kept=route[8:16], offsets=route[16:])
    return s


def test_output_is_the_layers(step):
    D = step.L.dev
    want = moe.layer_forward(step.cfg, D["x"], *step.weights, logit_bias=D["bias"])
    assert torch.equal(step.out, want)
    assert moe.get_device_error() == 0


def test_routing_in_the_checkpoint(step):
    D, k = step.L.dev, step.kept
    idx, w, lg = moe.router_topk(step.cfg, D["x"], D["wr"], D["bias"], want_logits=True)
    assert np.array_equal(k["topk_idx"], idx.cpu().numpy()) and np.array_equal(k["topk_w"], w.cpu().numpy())
    assert np.array_equal(k["logits"], lg.cpu().numpy())
    disp = moe.dispatch(step.cfg, D["x"], idx, w, gather=False)
    n = int(k["offsets"][8])
    for name in ("counts_raw", "counts_kept", "offsets", "slot_of"):
        assert np.array_equal(k[name], disp[name].cpu().numpy()), name
    for name in ("perm", "row_scale"):
        assert np.array_equal(k[name][:n], disp[name].cpu().numpy()[:n]), name


def _preacts(s, name, codes, scale):
    """Exact pre-activations of the kept slots, their summed magnitudes, and the decoded ones."""
    k, x = s.kept, oracle.to_f64(s.L.x)
    n = int(k["offsets"][8])
    want, mag = np.zeros((n, s.w.f)), np.zeros((n, s.w.f))
    for e in range(8):
        r = slice(int(k["offsets"][e]), int(k["offsets"][e + 1]))
        rows, wt = x[k["perm"][r]], oracle.to_f64(getattr(s.L, name)[e])
        want[r], mag[r] = rows @ wt, np.abs(rows) @ np.abs(wt)
    return want, mag, oracle.decode8(k[codes][:n], k[scale][:n])


@pytest.mark.parametrize("name,codes,scale", [("wg", "g_codes", "g_scale"), ("wu", "u_codes", "u_scale")])
def test_codes_are_within_half_a_step(step, name, codes, scale):
    want, mag, got = _preacts(step, name, codes, scale)
    n = want.shape[0]
    s = np.repeat(step.kept[scale][:n].astype(np.float64), 32, axis=1)
    e = (step.w.d + 2) * 2.0 ** -23 * mag
    assert np.all(np.abs(got - want) <= e + 0.5 * s * (1 + 2.0 ** -6))
    amax = np.repeat(np.abs(want).reshape(n, -1, 32).max(2), 32, axis=1)
    emax = np.repeat(e.reshape(n, -1, 32).max(2), 32, axis=1)
    assert np.all(np.abs(s - amax / 127) <= emax / 127 + 2.0 ** -8 * amax / 127)
    assert np.abs(step.kept[codes][:n]).max() <= 127


def _bounds(s, g, u, ref):
    """Entry by entry, the bound stated at the top."""
    k, w = s.kept, s.w
    x, wr, go = (np.abs(oracle.to_f64(v)) for v in (s.L.x, s.L.wr, s.go))
    b, t = 2.0 ** -8, lambda n: (n + 2) * 2.0 ** -23
    dwt_err, dx_err = np.zeros((w.T, 2)), np.zeros((w.T, w.d))
    dx_mag, lim = np.zeros((w.T, w.d)), {q: np.zeros(ref[q].shape) for q in KEYS}
    for e in range(8):
        wg, wu, wd = (np.abs(oracle.to_f64(getattr(s.L, q)[e])) for q in ("wg", "wu", "wd"))
        ts, js = np.nonzero((k["topk_idx"] == e) & (k["slot_of"] >= 0))
        r = k["slot_of"][ts, js]
        if not r.size:
            continue
        gg, uu = g[r], np.abs(u[r])
        sig = 1 / (1 + np.exp(-gg))
        sp, sl = sig * (1 + np.abs(gg) * (1 - sig)), np.abs(gg) * sig
        h = sl * uu
        dhu = np.abs(oracle.to_f64(s.go)[ts] @ oracle.to_f64(s.L.wd[e]).T)
        eh = t(w.d) * (go[ts] @ wd.T)
        wt = k["topk_w"][ts, js][:, None].astype(np.float64)
        dg, du = wt * dhu * uu * sp, wt * dhu * sl
        eg, eu = wt * uu * sp * eh + (b + 2.0 ** -16) * dg, wt * sl * eh + (b + 2.0 ** -16) * du
        lim["dw_gate"][e] = x[ts].T @ (eg + t(r.size) * (dg + eg))
        lim["dw_up"][e] = x[ts].T @ (eu + t(r.size) * (du + eu))
        lim["dw_down"][e] = (wt * h * (b + 2.0 ** -16 + t(r.size) * (1 + b))).T @ go[ts]
        np.add.at(dx_err, ts, eg @ wg.T + eu @ wu.T)
        np.add.at(dx_mag, ts, (dg + eg) @ wg.T + (du + eu) @ wu.T)
        dwt_err[ts, js] = np.sum(eh * h + (t(w.f) + 2.0 ** -16) * (dhu + eh) * h, axis=1)
    wt = k["topk_w"].astype(np.float64)
    mean = np.sum(wt * dwt_err, 1, keepdims=True)
    mag = np.abs(ref["dweight"]) + np.sum(wt * np.abs(ref["dweight"]), 1, keepdims=True)
    per = wt * (dwt_err + mean + 2.0 ** -20 * mag)
    dle = 2.0 ** -22 * np.abs(s.aux.astype(np.float64))
    for j in range(2):
        np.add.at(dle, (np.arange(w.T), k["topk_idx"][:, j]), per[:, j])
    dl = np.abs(ref["dlogits"]) + dle
    lim["dx"] = dx_err + t(2 * w.f + 10) * (dx_mag + dl @ wr) + dle @ wr
    lim["dw_router"] = dle.T @ x + t(w.T) * (dl.T @ x)
    lim["dbias"] = dle.sum(0) + t(w.T) * dl.sum(0)
    return {q: (1 + b) * v + b * np.abs(ref[q]) + 1e-30 for q, v in lim.items()}


def test_gradients_within_their_bounds(step):
    s, k = step, step.kept
    g, u = _preacts(s, "wg", "g_codes", "g_scale")[2], _preacts(s, "wu", "u_codes", "u_scale")[2]
    ref = oracle.layer_backward_at(s.L.x, s.L.wr, s.L.wg, s.L.wu, s.L.wd, s.go, k["topk_idx"], k["topk_w"],
                                   k["slot_of"], g, u, s.aux)
    lim = _bounds(s, g, u, ref)
    for q in KEYS:
        assert s.grads[q].dtype == torch.bfloat16 and s.grads[q].shape == ref[q].shape
        err = np.abs(to_np64(s.grads[q]) - ref[q])
        assert np.all(err <= lim[q]), (q, float(np.max(err / lim[q])))
    used = set(np.asarray(k["topk_idx"])[np.asarray(k["slot_of"]) >= 0].tolist())
    for e in set(range(8)) - used:
        for q in ("dw_gate", "dw_up", "dw_down"):
            assert not s.grads[q][e].any(), (q, e)
    assert moe.get_device_error() == 0


def test_backward_again_and_without_the_options(step):
    s = step
    aux = torch.from_numpy(s.aux).cuda()
    before = s.ck.clone()
    given = {q: torch.full_like(t, 3.0) for q, t in s.grads.items()}
    again = s.backward(dlogits=aux, grads=given)
    for q in KEYS:
        assert again[q] is given[q] and torch.equal(again[q], s.grads[q]), q
    assert torch.equal(before, s.ck)
    zero = s.backward(dlogits=torch.zeros_like(aux))
    none = s.backward(want_dbias=False)
    assert none["dbias"] is None
    for q in ("dw_gate", "dw_up", "dw_down"):
        assert torch.equal(zero[q], none[q]) and torch.equal(zero[q], s.grads[q]), q


def test_shared_scratch_of_two_layers_and_a_replayed_graph():
    """Two layers with a checkpoint each and one scratch, a balance loss on both, captured and replayed on new input."""
    a, b = Step("ragged"), Step("ragged", dict(capacity_factor=4.0))
    b.ws = a.ws
    go = to_dev(a.go)

    def run():
        res = []
        o1 = a.forward()
        o2 = moe.layer_forward_train_c8(b.cfg, o1, *b.weights, b.ck, b.ws)
        v = moe.checkpoint_views_c8(b.cfg, b.ck)
        loss = moe.balance_loss(b.cfg, v["logits"], v["topk_idx"], z_coef=0.01)
        g2 = moe.layer_backward_c8(b.cfg, o1, *b.weights, go, b.ck, b.ws, dlogits=loss["dlogits"])
        g1 = moe.layer_backward_c8(a.cfg, a.L.dev["x"], *a.weights, g2["dx"], a.ck, a.ws)
        res += [o2, loss["loss"], loss["counts"]] + [g2[q] for q in KEYS] + [g1[q] for q in KEYS]
        return res

    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = run()
    for call in (3, 4):
        a.L.dev["x"].copy_(to_dev(configs.make_x(a.w, call=0) if call == 3 else normal(5, 77, (a.w.T, a.w.d), dtype="bf16")))
        graph.replay()
        got = [t.clone() for t in captured]
        want = run()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(got, want)):
            assert torch.equal(p, q), i
    assert moe.get_device_error() == 0


def test_checkpoint_at_a_16_byte_address():
    """The alignment that every buffer of the library may have gives the same bits."""
    s = Step("ragged")
    out, grads = s.forward(), s.backward()
    s.ck = torch.empty(s.ck.numel() + 16, dtype=torch.uint8, device="cuda")[16:]
    assert s.ck.data_ptr() % 32 == 16
    assert torch.equal(out, s.forward())
    again = s.backward()
    for q in KEYS:
        assert torch.equal(grads[q], again[q]), q
    assert moe.get_device_error() == 0


def test_tile_mode_does_not_change_the_bits():
    s = Step("ragged")
    out, grads = s.forward(), s.backward()
    with moe.gemm_tiles("pair"):
        assert torch.equal(out, s.forward())
        again = s.backward()
    for q in KEYS:
        assert torch.equal(grads[q], again[q]), q
    assert moe.get_device_error() == 0


def test_two_steps_on_two_streams_at_once():
    steps = [Step("ragged"), Step("drop"), Step("two_experts")]
    want = [(s.forward(), s.backward()) for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [[] for _ in steps]
    for _ in range(3):
        for s, st, g in zip(steps, streams, got):
            with torch.cuda.stream(st):
                g.append((s.forward(), s.backward()))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for out, grads in g:
            assert torch.equal(w[0], out)
            for q in KEYS:
                assert torch.equal(w[1][q], grads[q]), q
    assert moe.get_device_error() == 0


def test_offsets_past_32_bits():
    """140000 rows of 32768 columns: more than 2^32 codes and values.  A token's output and dx depend on its own row
    alone, so the last tokens' equal those of a batch of them, and the rest's weight gradients add up."""
    T, n, d, f = 70000, 600, 256, 32768
    gen = torch.Generator(device="cuda").manual_seed(11)

    def normal_(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(std=std, generator=gen)

    x, dout = normal_(T, d), normal_(T, d)
    weights = (normal_(8, d, std=d ** -0.5), normal_(8, d, f, std=d ** -0.5), normal_(8, d, f, std=d ** -0.5),
               normal_(8, f, d, std=f ** -0.5))

    def step(lo, hi):
        c = moe.Config(hi - lo, d, f, capacity_factor=4.0)
        ck, ws = _buffers(c)
        out = moe.layer_forward_train_c8(c, x[lo:hi], *weights, ck, ws)
        return out, moe.layer_backward_c8(c, x[lo:hi], *weights, dout[lo:hi], ck, ws)

    out, g = step(0, T)
    last, gl = step(T - n, T)
    assert torch.equal(out[T - n:], last) and torch.equal(g["dx"][T - n:], gl["dx"])
    first, gf = step(0, T - n)
    assert torch.equal(out[:T - n], first)
    for q in KEYS[3:]:
        # three bf16 roundings; and on both sides fp32 sums of the same n = 17500 terms an expert, off by at most
        # (n + 2) 2^-23 sum |term|, where sum |term| is about 0.8^2 sqrt(n) = 84 times the sum's rms (130 taken)
        got, want = g[q].float(), gf[q].float() + gl[q].float()
        tol = 3 * 2.0 ** -9 * (gf[q].float().abs() + gl[q].float().abs() + got.abs()) + 0.54 * got.pow(2).mean().sqrt()
        assert ((got - want).abs() <= tol).all(), q
    assert moe.get_device_error() == 0


def test_blocks_with_overflow_and_zero_rows():
    s = Step("few_rows")
    x = s.L.dev["x"]
    x[7] = 0
    x[9] = 3e38  # its pre-activations pass fp32's range
    out = s.forward()
    torch.cuda.synchronize()
    v = moe.checkpoint_views_c8(s.cfg, s.ck)
    n = int(v["route"][24])
    tok = v["perm"][:n]
    for q in ("g", "u"):
        scale, codes = v[q + "_scale"][:n].float(), v[q + "_codes"][:n]
        assert not scale[tok == 7].any() and not codes[tok == 7].any()
        bad = torch.isnan(scale[tok == 9])
        assert bad.any() and not codes[tok == 9].view(-1, s.w.f // 32, 32)[bad].any()
        assert torch.isfinite(scale[(tok != 9)]).all()
    rest = torch.ones(s.w.T, dtype=torch.bool)
    rest[9] = False
    assert torch.isfinite(out[rest.cuda()].float()).all() and not out[7].any()
    assert moe.get_device_error() == 0


def test_no_tokens_gives_zero_gradients():
    cfg = moe.Config(0, 256, 256)
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ws = (z(8, 256), z(8, 256, 256), z(8, 256, 256), z(8, 256, 256))
    ck, sc = _buffers(cfg)
    out = moe.layer_forward_train_c8(cfg, z(0, 256), *ws, ck, sc)
    assert out.shape == (0, 256)
    grads = {q: torch.full((8, 256, 256), 2.0, dtype=torch.bfloat16, device="cuda") for q in KEYS[3:]}
    g = moe.layer_backward_c8(cfg, z(0, 256), *ws, z(0, 256), ck, sc, grads=grads)
    for q in KEYS:
        assert not g[q].any(), q


@pytest.mark.parametrize("T", [60, 700])
def test_bf16_pair_takes_the_balance_gradient(T):
    """layer_backward with dlogits: dx and dw_router move by dlogits W_r and dlogits^T x, the experts' gradients not at all."""
    w = configs.scaled(W["mid_bf16"], name="aux", T=T, d=256, f=256, capacity_factor=1.25)
    L = LayerInputs(w)
    D = L.dev
    ws = torch.empty(moe.workspace_size_train(L.cfg), dtype=torch.uint8, device="cuda")
    moe.layer_forward_train(L.cfg, D["x"], D["wr"], D["wg"], D["wu"], D["wd"], ws)
    go = to_dev(normal(configs.SEED, 907, (T, 256), dtype="bf16"))
    idx, _, lg = moe.router_topk(L.cfg, D["x"], D["wr"], want_logits=True)
    dl = moe.balance_loss(L.cfg, lg, idx, balance_coef=30.0, z_coef=5.0)["dlogits"]
    args = (L.cfg, D["x"], D["wr"], D["wg"], D["wu"], D["wd"], go, ws)
    old, new = moe.layer_backward(*args), moe.layer_backward(*args, dlogits=dl)
    for q in ("dw_gate", "dw_up", "dw_down"):
        assert torch.equal(old[q], new[q]), q
    dl64, x64, wr64 = to_np64(dl), to_np64(D["x"]), to_np64(D["wr"])
    t = (T + 2) * 2.0 ** -23
    mag = np.abs(to_np64(old["dw_router"])) + np.abs(dl64).T @ np.abs(x64)
    # both sides' sums of T fp32 terms; the softmax part's terms are within the magnitudes of the first
    soft = oracle.layer_backward(L.x, L.wr, L.wg, L.wu, L.wd, 1.25, normal(configs.SEED, 907, (T, 256), dtype="bf16"))
    mag += 1.1 * np.abs(soft["dlogits"]).T @ np.abs(x64)
    assert np.all(np.abs(to_np64(new["dw_router"]) - to_np64(old["dw_router"]) - dl64.T @ x64) <= 2 * t * mag)
    change = to_np64(new["dx"]) - to_np64(old["dx"])
    b = 2.0 ** -8
    lim = b * (np.abs(to_np64(new["dx"])) + np.abs(to_np64(old["dx"]))) * 1.01 + 2.0 ** -18 * (np.abs(dl64) @ np.abs(wr64) + np.abs(to_np64(old["dx"])))
    assert np.all(np.abs(change - dl64 @ wr64) <= lim)
    assert moe.get_device_error() == 0
