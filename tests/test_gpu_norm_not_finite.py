"""ss_rmsnorm_act of rows that are not finite (a NaN or an infinity in x, in the sum of finite values, in the weights, products
beyond float32), among rows that are: bit for bit the oracle's, where a NaN is a NaN, in every form of the kernel."""
import numpy as np
import pytest
import torch

import oracle
from helpers import dev_bf16, dev_f32, have_gpu, host
from oracle.norm import codes, rmsnorm
from oracle.quant import f32_to_bf16_rne

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

SIZES = [8, 100, 130, 500, 777, 2048, 4096, 8000, 16384, 17000, 33000]  # threads a row 16, 64, 256 .. 1024, and rows over memory


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


def _dev(x, bf16):
    pad = np.zeros((x.shape[0], (x.shape[1] + 7) // 8 * 8), np.float32)
    pad[:, : x.shape[1]] = x
    return (dev_bf16(oracle.f32_to_bf16_bits_rne(pad)) if bf16 else dev_f32(pad))[:, : x.shape[1]]


def _same(got, exp):
    got = got.float().cpu().numpy()
    return np.array_equal(got, exp, equal_nan=True)


def _check(ss, x, w, eps, res, bf16, n=2):
    z, r = rmsnorm(x, w, eps, res, bf16)
    tx, tr, tw = _dev(x, bf16), None if res is None else _dev(res, bf16), None if w is None else dev_f32(w)
    y, sx, total = ss.rmsnorm_act(tx, tw, eps, residual=tr)
    assert sx is None and _same(y, f32_to_bf16_rne(z))
    assert total is None or _same(total, r)
    for q in ("i8", "fp8"):
        y, sx, total = ss.rmsnorm_act(tx, tw, eps, residual=tr, n=n, y_dtype=q)
        c, s = codes(z, n, q)
        assert _same(sx, s) and np.array_equal(host(y), c)
    return z


@pytest.mark.parametrize("K", SIZES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n", [2, 4, 5])
def test_not_finite_values_of_a_row(ss, K, bf16, n):
    rng = np.random.default_rng(K)
    x = rng.standard_normal((7, K)).astype(np.float32)
    res = rng.standard_normal((7, K)).astype(np.float32)
    if bf16:
        x, res = f32_to_bf16_rne(x), f32_to_bf16_rne(res)
    big = f32_to_bf16_rne(np.float32([3e38]))[0]
    x[0, K - 1] = np.nan
    x[1, K // 2] = np.inf
    x[3, 0], x[3, K - 1] = -np.inf, np.nan
    x[4, K - 1] = res[4, K - 1] = big  # finite, the sum is not
    x[5, 0], res[5, 0] = np.inf, -np.inf
    w = (0.1 + rng.random(K)).astype(np.float32)
    for weights in (w, None):
        z = _check(ss, x, weights, 1e-5, res, bf16, n)
        assert np.isnan(z[[0, 3, 5]]).all() and np.isnan(z[[1, 4]]).sum() == 2 and np.isfinite(z[[2, 6]]).all()
        z = _check(ss, x[[0, 1, 2, 3]], weights, 0.0, None, bf16, n)
        assert np.isnan(z[[0, 3]]).all() and np.isnan(z[1]).sum() == 1 and np.isfinite(z[2]).all()


@pytest.mark.parametrize("K", SIZES)
@pytest.mark.parametrize("at,value", [(0, np.nan), (-1, np.nan), (0, np.inf), (-1, -np.inf), (-1, 3e38)])
def test_not_finite_weights(ss, K, at, value):
    rng = np.random.default_rng(K)
    x = rng.standard_normal((5, K)).astype(np.float32)
    x[1] = 0  # 0 w: NaN for weights that are not finite
    x[2, at], x[3, at] = 0, 1
    x[4] = 0
    x[4, at] = 5.0  # z = sqrt(K): beyond float32 times 3e38
    w = (0.1 + rng.random(K)).astype(np.float32)
    w[at] = value
    z = _check(ss, x, w, 0.0, None, False)
    assert np.isfinite(z[:, : K // 2 if at else 0]).all() and not np.isfinite(z[4, at])


@pytest.mark.parametrize("K", SIZES)
def test_roots_beyond_float32(ss, K):
    x = np.zeros((4, K), np.float32)
    x[0, 0], x[1, K - 1], x[2] = 1e-40, -3e-42, 1e-44
    _check(ss, x, None, 0.0, None, False)


def test_a_row_with_a_nan_has_products_of_nan(ss):
    """Scale and codes through the sparse product: NaN all over the token's row, the other tokens as without it."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((20, 512), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn((256, 512), generator=g, device="cuda")
    for q in ("i8", "fp8"):
        vals, meta, sw = ss.slide_decompose(W, 4, q)

        def out(t):
            y, sx, _ = ss.rmsnorm_act(t, None, 1e-6, n=4, y_dtype=q)
            return ss.spgemm(ss.SS_SPARSE_W, 20, 256, y.shape[1], vals, meta, y, sx=sx, sw=sw)

        clean = out(x)
        bad = x.clone()
        bad[7, 100], bad[11, 3] = float("nan"), float("inf")
        got = out(bad)
        rows = torch.tensor([i not in (7, 11) for i in range(20)], device="cuda")
        assert got.shape[0] == 20 and torch.equal(got[rows], clean[rows]) and got[~rows].isnan().all()
