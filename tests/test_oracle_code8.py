"""The oracle's 8-bit activation codes and its backward at given pre-activations."""
import numpy as np

import oracle


def test_codes_stay_within_half_a_step():
    r = np.random.default_rng(0)
    v = r.normal(0, 1, (40, 96)) * 10.0 ** r.integers(-30, 30, (40, 1))
    v[3, 32:64] = 0
    v[4, :32] = 1e-41
    c, s = oracle.code8(v)
    assert np.abs(c).max() <= 127 and c[3, 32:64].max() == 0 and s[3, 1] == 0 and s[4, 0] == 0
    step = np.repeat(s, 32, axis=1)
    # the clipped end: amax / s <= 127 / (1 - 2^-8) < 127.5, so rint never leaves the codes
    live = step > 0
    assert np.all(np.abs(oracle.decode8(c, s) - v)[live] <= 0.5 * step[live] * (1 + 1e-12))
    v[5, 40] = np.nan
    v[6, 0] = -np.inf
    c, s = oracle.code8(v)
    assert np.isnan(s[5, 1]) and np.isnan(s[6, 0]) and not c[5, 32:64].any() and np.isfinite(s[5, [0, 2]]).all()


def test_backward_at_the_exact_preactivations_is_the_layer_backward_and_the_differences():
    r = np.random.default_rng(1)
    T, d, f = 12, 8, 32
    x, dout = r.normal(0, 1, (T, d)), r.normal(0, 1, (T, d))
    wr, wg, wu, wd = (r.normal(0, 0.4, s) for s in ((8, d), (8, d, f), (8, d, f), (8, f, d)))
    want = oracle.layer_backward(x, wr, wg, wu, wd, 1.25, dout)
    idx, w, slot = want["idx"], want["w"], want["slot_of"]
    n = want["n_kept"]
    g, u = np.zeros((n, f)), np.zeros((n, f))
    for t in range(T):
        for j in range(2):
            if slot[t, j] >= 0:
                g[slot[t, j]], u[slot[t, j]] = x[t] @ wg[idx[t, j]], x[t] @ wu[idx[t, j]]
    got = oracle.layer_backward_at(x, wr, wg, wu, wd, dout, idx, w, slot, g, u)
    for k in ("dx", "dw_router", "dbias", "dw_gate", "dw_up", "dw_down", "dweight"):
        assert np.allclose(got[k], want[k], rtol=1e-12, atol=1e-12), k
    aux = r.normal(0, 1, (T, 8))
    more = oracle.layer_backward_at(x, wr, wg, wu, wd, dout, idx, w, slot, g, u, aux)
    assert np.allclose(more["dx"] - got["dx"], aux @ wr) and np.allclose(more["dw_router"] - got["dw_router"], aux.T @ x)

    # against central differences of sum(out dout) + sum(aux logits) along a direction of every input
    def value(h, dirs):
        a = [p + h * q for p, q in zip((x, wr, wg, wu, wd), dirs)]
        return float(np.sum(oracle.layer_forward(*a, 1.25)["out"] * dout) + np.sum(aux * (a[0] @ a[1].T)))

    dirs = [r.normal(0, 1, v.shape) for v in (x, wr, wg, wu, wd)]
    h = 1e-6
    slope = (value(h, dirs) - value(-h, dirs)) / (2 * h)
    along = sum(float(np.sum(more[k] * q)) for k, q in zip(("dx", "dw_router", "dw_gate", "dw_up", "dw_down"), dirs))
    assert abs(slope - along) <= 1e-6 * max(1.0, abs(along))
