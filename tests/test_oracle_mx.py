"""The oracle's microscaled formats against the format's own tables."""
import numpy as np
import torch

import oracle


def test_e2m1_rounds_to_the_nearest_code_and_ties_to_even():
    for a, want in [(0.25, 0), (0.26, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (5.1, 7), (6.9, 7)]:
        w = np.zeros((32, 1))
        w[0], w[1], w[2] = 4.0, a, -a  # 4 sets the scale to 1 ...
        codes, x = oracle.mx4_blocks(w)
        if a > 4:
            assert x[0, 0] == 0  # ... and so does anything up to 7
        assert x[0, 0] == 0 and codes[1, 0] == want and codes[2, 0] == want + 8, a


def test_scale_rule():
    assert [int(oracle.mx_exponent(v, 2, 125)) for v in (4.0, 7.0, 7.01, 8.0, 0.0, 3.3e38, 1e-40)] == [0, 0, 1, 1, -127, 125, -127]
    w = np.zeros((64, 2))
    w[3, 0], w[40, 1] = np.nan, np.inf
    codes, x = oracle.mx4_blocks(w)
    assert x[0, 0] == 128 and x[1, 1] == 128 and x[0, 1] == x[1, 0] == -127 and not codes.any()


def test_e4m3_agrees_with_the_type():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = oracle.e4m3_values(np.arange(256))
    assert np.array_equal(got, v, equal_nan=True)
    r = np.random.default_rng(0).normal(0, 1, 4000) * 2.0 ** np.random.default_rng(1).integers(-14, 8, 4000)
    r = np.clip(r, -448, 448)
    want = torch.from_numpy(r).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_round(r.astype(np.float32).astype(np.float64)), want)


def test_packing_and_values():
    r = np.random.default_rng(2)
    w = r.normal(0, 1, (256, 128))
    codes, x = oracle.mx4_blocks(w)
    q, s = oracle.mx4_pack(codes, x)
    assert q.shape == (128, 128) and s.shape == (1, 2, 512)
    assert q[5, 7] & 15 == codes[14, 5] and q[5, 7] >> 4 == codes[15, 5]
    assert s[0, 1, (70 % 32) * 16 + 70 // 32 * 4 + 2] == x[6, 70] + 127
    v = oracle.mx4_values(codes, x)
    step = np.repeat(np.ldexp(1.0, x), 32, axis=0)
    # half of the widest step (2), and up to 1 where the block's largest element is between 6 and 7
    assert np.all(np.abs(v - w) <= step) and np.mean((v - w) ** 2) < 0.02
