"""What the microscaled 8-bit rows are stated to lose, on rows whose blocks span many powers of two."""
import numpy as np

import oracle


def test_e4m3_rows_lose_a_sixteenth_or_a_step_of_the_smallest_elements():
    r = np.random.default_rng(4)
    v = r.normal(0, 1, (300, 128)) * 2.0 ** r.integers(-24, 1, (300, 128))
    got, x = oracle.mx8_rows(v)
    unit = np.repeat(np.ldexp(1.0, x), 32, axis=1)
    err = np.abs(got - v)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * unit))
    # the second term is needed: elements under 2^-10 of the scale are lost whole
    small = np.abs(v) < 2.0 ** -10 * unit
    assert small.any() and not got[small].any()
    assert np.all(err[np.abs(v) >= 2.0 ** -6 * unit] <= 2.0 ** -4 * np.abs(v[np.abs(v) >= 2.0 ** -6 * unit]))
