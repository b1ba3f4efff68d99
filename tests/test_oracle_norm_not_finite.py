"""Pins of the norm's oracle for rows that are not finite, and for roots beyond float32."""
import numpy as np

from oracle.norm import codes, rmsnorm

BIG = np.float32(3e38)


def test_a_nan_is_all_over_its_row_and_an_infinity_in_its_place():
    x = np.array([[1, np.nan, 2], [1, np.inf, 2], [-np.inf, 1, 0], [3, -4, 0]], np.float32)
    z, _ = rmsnorm(x, None, 0.0, bf16=False)
    assert np.isnan(z).tolist() == [[True] * 3, [False, True, False], [True, False, False], [False] * 3]
    assert z[1, 0] == 0 and z[2, 1] == 0
    z, r = rmsnorm([[BIG, 1]], None, 1e-6, [[BIG, 1]], bf16=False)  # finite values whose sum is not
    assert np.isinf(r[0, 0]) and np.isnan(z[0, 0]) and z[0, 1] == 0


def test_codes_of_rows_that_are_not_finite():
    z = np.array([[1, np.nan, 2, 0], [1, -np.inf, 2, 0], [0, 0, 0, 0], [1, 2, -4, 0]], np.float32)
    for q in ("i8", "fp8"):
        c, s = codes(z, 2, q)
        assert (c[:3] == 0).all() and (c[3, :3] != 0).all()
        assert np.isnan(s[0]) and np.isposinf(s[1]) and s[2] == 0 and s[3] > 0


def test_roots_beyond_float32():
    z, _ = rmsnorm([[1e-40, 0, 0, 0]], None, 0.0, bf16=False)  # 1 / sqrt(1e-80 / 4) = 2e40
    assert np.isfinite(z).all() and z[0, 0] == np.float32(1e-40) * np.finfo(np.float32).max and (z[0, 1:] == 0).all()
