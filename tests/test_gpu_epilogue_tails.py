"""The activations of ss_spgemm_tiled_epilogue far from zero, relative to their values."""
import math

import numpy as np
import pytest
import torch

from helpers import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


@pytest.mark.parametrize("M,N", [(3, 514), (40, 514), (300, 514), (300, 515), (2200, 4096)])
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_gelu_relative_to_its_value(ss, M, N, y):
    """gelu(z) = z Phi(z) falls to 1e-32 at z = -12 without losing its bits. The product is zero, so z is the bias.
    The argument of the complementary error function, x = -z / sqrt 2, rounds by 2^-23 (constant and product), which
    moves erfc(x) by x erfc'(x) / erfc(x) of that, at most 2 x^2 + 2 = z^2 + 2 times; its square and the exponent's
    product round by 2^-24 of z^2 / 2 log2 e each, the power's argument; the function itself is good to 2^-16
    (bf16 results) or 2^-20 (f32), and what follows rounds by 2^-22 at most."""
    Kc = 256
    W = torch.randn((N, Kc), device="cuda")
    v, m, sw = ss.slide_decompose(W, 2, "i8")
    tv, tm = ss.pack_sparse(v, m)
    dense, sx = torch.zeros((M, Kc), dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda")
    z = torch.linspace(-12, 7, N, device="cuda")
    got = ss.spgemm_tiled_epilogue(ss.SS_SPARSE_W, M, N, Kc, tv, tm, dense, sx, sw, bias=z, act="gelu", y_dtype=y)
    zd = z.double().cpu().numpy()
    want = np.array([t / 2 * math.erfc(-t / math.sqrt(2)) for t in zd])
    rel = (zd ** 2 + 2) * 2.0 ** -23 + zd ** 2 * 2.0 ** -23 + (2.0 ** -16 if y == "bf16" else 2.0 ** -20) + 2.0 ** -22
    rel = rel + (2.0 ** -8 if y == "bf16" else 2.0 ** -24) * (1 + rel)
    err = np.abs(got.double().cpu().numpy() - want) / np.maximum(np.abs(want), 1e-300)
    assert (err <= rel).all(), (float((err / rel).max()), zd[int((err / rel).max(0).argmax())])
