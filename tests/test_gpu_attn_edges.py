"""ss_attn where a tile's rows share one token (32 query heads and more to a key head), for every form of the kernels:
tiles of many rows, the keys in two parts, few rows in one workgroup and in several."""
import pytest
import torch

from helpers import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


@pytest.mark.parametrize("G", [32, 33, 40, 48, 64, 71])
@pytest.mark.parametrize("lq,lk,D", [
    (20, 60, 128), (20, 75, 64), (30, 25, 72),  # tiles of many rows
    (200, 600, 64), (200, 1100, 128),  # the keys in two parts
    (6, 500, 128), (2, 40, 64),  # few rows, one workgroup
    (6, 5000, 128), (3, 2500, 64)])  # and several
def test_infinities_and_nan_with_a_token_per_tile(ss, lq, lk, D, G):
    """Values that are infinite or NaN reach the rows that see them, and leave every bit of the others alone."""
    g = torch.Generator(device="cuda").manual_seed(lq + G)
    q = torch.randn((lq, G, D), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((lk, 1, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    lse, lse_k = (torch.empty((G, lq), device="cuda") for _ in range(2))
    clean = ss.attn(q, k, v, lse=lse)
    assert clean.isfinite().all()
    seen = (torch.arange(lq, device="cuda") + lk - lq + 1).clamp(0, lk)  # keys of a row
    for back in sorted({1, 2, min(lq - 1, 5), min(lq - 1, 40)}):
        j = max(lk - back, 0)
        rows = seen > j
        vb = v.clone()
        vb[j, :, 1], vb[j, :, 3], vb[j, :, D - 1] = float("nan"), float("inf"), -float("inf")
        o = ss.attn(q, k, vb, lse=lse_k)
        assert torch.equal(o[~rows], clean[~rows]) and torch.equal(lse_k, lse)
        other = [c for c in range(D) if c not in (1, 3, D - 1)]
        assert torch.equal(o[:, :, other], clean[:, :, other])
        assert o[rows][:, :, 1].isnan().all() and (o[rows][:, :, 3] == float("inf")).all()
        assert (o[rows][:, :, D - 1] == -float("inf")).all()
        kb = k.clone()
        kb[j, :, 2] = float("nan")
        o = ss.attn(q, kb, v, lse=lse_k)
        assert torch.equal(o[~rows], clean[~rows]) and torch.equal(lse_k[:, ~rows], lse[:, ~rows])
        assert o[rows].isnan().all() and lse_k[:, rows].isnan().all()
