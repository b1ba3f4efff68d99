"""Pins of the oracles of the norm, the windowed and the paged attention."""
import numpy as np

from oracle.attention import attention
from oracle.norm import codes, rmsnorm
from oracle.quant import quant_rows
from oracle.windowed import attend, packed, paged, seen


def test_norm_of_known_rows():
    z, r = rmsnorm([[3.0, -4.0], [0.0, 0.0]], [2.0, 1.0], eps=0.0, bf16=False)
    rms = np.sqrt(12.5)
    assert np.allclose(z[0], [6 / rms, -4 / rms], rtol=1e-6) and (z[1] == 0).all()
    z, r = rmsnorm([[1.0, 1.0]], None, 3.0, [[1.0 + 2.0 ** -9, 0.0]], bf16=True)
    assert (r == [[2.0, 1.0]]).all()  # 2 + 2^-9 rounds to 2 in bf16
    assert np.allclose(z, np.array([[2.0, 1.0]]) / np.sqrt(5.5), rtol=1e-6)


def test_codes_are_the_quantisers_but_for_borders():
    z = np.random.default_rng(0).standard_normal((300, 256)).astype(np.float32)
    c, s = codes(z, 2, "i8")
    c2, s2 = quant_rows(z, "i8")
    assert np.array_equal(s, s2) and np.abs(c.astype(int) - c2).max() <= 1
    t = z.astype(np.float64) * 127 / np.abs(z).max(1, keepdims=True)
    assert (np.abs(t - np.floor(t) - 0.5)[c != c2] <= 127 * 2.0 ** -22).all()
    z = z[:3]
    c, c2 = codes(z, 2, "i8")[0], quant_rows(z, "i8")[0]
    assert np.array_equal(c, c2)  # (no value of these rows lies at a border)
    c, _ = codes(z, 4, "i8")  # 6:8: windows 0-3, 2-5, 4-7 of a group
    assert np.array_equal(c[:, :12], c2[:, [0, 1, 2, 3, 2, 3, 4, 5, 4, 5, 6, 7]]) and c.shape[1] == 512


def test_what_a_window_shows():
    see = seen(3, 6, True, 2, 1)
    assert see.astype(int).tolist() == [[1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert seen(3, 2, True).sum(1).tolist() == [0, 1, 2] and seen(2, 3, False).all()


def test_without_a_window_it_is_the_packed_attention():
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal((9, 4, 8)), r.standard_normal((13, 2, 8)), r.standard_normal((13, 2, 8))
    for x, y in zip(attention(q, k, v, [0, 3, 7], [0, 5, 12], [4, 7]), packed(q, k, v, [0, 3, 7], [0, 5, 12], [4, 7])):
        assert np.allclose(x, y, equal_nan=True)


def test_pages_are_the_keys_in_order():
    r = np.random.default_rng(2)
    kp, vp = r.standard_normal((5, 4, 1, 8)), r.standard_normal((5, 4, 1, 8))
    q = r.standard_normal((1, 2, 8))
    table = [[3, 0, 9]]  # the last entry names no page
    k, v = np.concatenate([kp[3], kp[0]]), np.concatenate([vp[3], vp[0]])
    see = np.ones((1, 8), bool)
    for x, y in zip(paged(q, kp, vp, table, [11], [0, 1]), attend(q, k, v, see)):
        assert np.allclose(x, y)
    # a window of 5 from position 10 on, of which entry 2 holds three: keys 6 and 7 are left, and the first token
    see[0, 1:6] = False
    for x, y in zip(paged(q, kp, vp, table, [11], [0, 1], window=5, sinks=1), attend(q, k, v, see)):
        assert np.allclose(x, y)
