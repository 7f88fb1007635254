"""The oracle's balance loss against its definition: a balanced router gives 1,
the gradient agrees with central differences, masked rows count for nothing."""
import numpy as np

import oracle


def _case(T=23, seed=3):
    r = np.random.default_rng(seed)
    lg = r.normal(0, 1.5, (T, 8))
    idx = np.argsort(-lg, axis=1)[:, :2]
    mask = r.random(T) < 0.8
    return lg, idx, mask, [2, 2, 9, 15, 20]


def test_balanced_router_gives_one():
    T = 16
    idx = np.stack([np.arange(T) % 8, (np.arange(T) + 4) % 8], 1)
    loss, counts, dl = oracle.balance_loss(np.zeros((T, 8)), idx, balance_coef=1.0)
    assert np.all(counts == 4) and abs(loss[1] - 1.0) < 1e-14 and abs(loss[2] - np.log(8) ** 2) < 1e-13
    assert np.max(np.abs(dl)) < 1e-16


def test_gradient_agrees_with_differences():
    lg, idx, mask, off = _case()
    _, _, dl = oracle.balance_loss(lg, idx, mask, off, 0.3, 0.2)
    h = 1e-5
    for t in range(lg.shape[0]):
        for e in range(8):
            up, dn = lg.copy(), lg.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = (oracle.balance_loss(up, idx, mask, off, 0.3, 0.2)[0][0] -
                 oracle.balance_loss(dn, idx, mask, off, 0.3, 0.2)[0][0]) / (2 * h)
            # truncation h^2 |f'''| / 6 below 1e-10, cancellation 2^-53 |loss| / h below 1e-11
            assert abs(d - dl[t, e]) < 2e-10


def test_rows_that_do_not_count():
    lg, idx, mask, off = _case()
    want = oracle.balance_loss(lg, idx, mask, off, 0.3, 0.2)
    out = np.ones(len(mask), bool)
    out[2:20] = ~mask[2:20]
    lg2 = lg.copy()
    lg2[out] = np.nan
    got = oracle.balance_loss(lg2, idx, mask, off, 0.3, 0.2)
    for a, b in zip(want, got):
        assert np.array_equal(a, b)
    assert np.all(got[2][out] == 0) and got[1][0].sum() == 0
    empty = oracle.balance_loss(lg, idx, np.zeros(len(mask), bool), off, 0.3, 0.2)
    assert not empty[0].any() and not empty[1].any() and not empty[2].any()
