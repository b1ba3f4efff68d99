"""Tiled products whose dense operand has two rows 2^31 bytes and more apart (within the 4 GiB that the calls allow): the
row-block kernel of few tokens, plain and with an epilogue, the small tiles and the 256 x 128 tiles of sparse activations."""
import pytest
import torch

from helpers import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


@pytest.mark.parametrize("q", ["i8", "bf16"])
@pytest.mark.parametrize("side", ["W", "X"])
def test_dense_rows_far_apart(ss, side, q):
    Kc, R = 512, 100
    g = torch.Generator(device="cuda").manual_seed(1)
    sp = torch.randn((R, Kc), generator=g, device="cuda")
    if q == "i8":
        v, m, s_sp = ss.slide_decompose(sp, 2, q)
        near = torch.randint(-127, 128, (2, Kc), generator=g, device="cuda", dtype=torch.int8)
        s_dn = torch.rand(2, generator=g, device="cuda")
    else:
        v, m, _ = ss.slide_decompose(sp, 2, q)
        near, s_sp, s_dn = torch.randn((2, Kc), generator=g, device="cuda").to(torch.bfloat16), None, None
    tv, tm = ss.pack_sparse(v, m)
    apart = ((1 << 31) + 4096) // near.element_size()
    far = torch.zeros(apart + Kc, dtype=near.dtype, device="cuda").as_strided((2, Kc), (apart, 1))
    far.copy_(near)
    M, N, sx, sw = (2, R, s_dn, s_sp) if side == "W" else (R, 2, s_sp, s_dn)
    code = ss.SS_SPARSE_W if side == "W" else ss.SS_SPARSE_X
    for y in ("bf16", "f32"):
        want = ss.spgemm_tiled(code, M, N, Kc, tv, tm, near, sx, sw, y)
        assert want.abs().sum() > 0
        assert torch.equal(ss.spgemm_tiled(code, M, N, Kc, tv, tm, far, sx, sw, y), want)
        for kw in (dict(), dict(act="silu", gated=True), dict(residual=want)):
            e = [ss.spgemm_tiled_epilogue(code, M, N, Kc, tv, tm, d, sx, sw, y_dtype=y, **kw) for d in (near, far)]
            assert torch.equal(e[0], e[1])
