"""ss_attn where a tile's rows share one token (32 query heads and more to a key head) and where scores are large, for
every form of the kernels: tiles of many rows, the keys in two parts, few rows in one workgroup and in several."""
import numpy as np
import pytest
import torch

from helpers import have_gpu
from oracle.attention import attention

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


@pytest.mark.parametrize("top", [34, 60, 110, 121])
@pytest.mark.parametrize("lq,lk,Hq,Hkv,D", [
    (200, 333, 2, 1, 128), (90, 200, 3, 1, 64),  # tiles of many rows
    (700, 900, 2, 2, 64), (600, 1100, 2, 2, 128),  # the keys in two parts
    (6, 500, 4, 1, 128), (40, 2000, 2, 1, 64),  # few rows, one workgroup and several
    (4, 5000, 7, 1, 72)])
def test_finite_scores_of_any_size(ss, lq, lk, Hq, Hkv, D, top):
    """Scores of up to 2^top, so far apart that a row is the value of its largest score, exactly. The scores are
    exact: only the first value of q and k is not zero, q a power of two, k of 8 bits: 512 different values within 4
    powers of two, the other keys alike at the end that loses. The closest two, scaled, are 2^(top - 11) / sqrt(D) apart,
    2^19 or more, whose power is zero. With q > 0 the largest of large scores wins, with q < 0 the least far of
    scores that are all far below zero. The logarithm: the scale, its product with log2 e, the maximum and its product
    with ln 2 round by 2^-24 each, and so do the two constants."""
    rng = np.random.default_rng(lk + D)
    steps = np.array([(1 + m / 128) * 2.0 ** e for e in range(4) for m in range(128)])
    seen = np.arange(lk)[None, :] <= (np.arange(lq) + lk - lq)[:, None]
    for sign in (1.0, -1.0):
        b = np.full(lk, 1.0 if sign > 0 else 16.0)
        own = rng.permutation(lk)[: min(512, lk)]
        b[own] = rng.permutation(steps)[: len(own)]
        q, k = np.zeros((lq, Hq, D)), np.zeros((lk, Hkv, D))
        q[:, :, 0] = sign * 2.0 ** (top // 2)
        k[:, :, 0] = (b * 2.0 ** (top - 4 - top // 2))[:, None]
        s = np.where(seen, q[:, :1, 0] * k[:, 0, 0], -np.inf)
        assert ((s == s.max(1)[:, None]).sum(1) == 1).all()
        qt, kt = (torch.from_numpy(x).to("cuda", torch.bfloat16) for x in (q, k))
        v = torch.from_numpy(rng.standard_normal((lk, Hkv, D))).to("cuda", torch.bfloat16)
        lse = torch.empty((Hq, lq), device="cuda")
        o = ss.attn(qt, kt, v, lse=lse)
        assert torch.equal(o, v[torch.from_numpy(s.argmax(1)).cuda()].repeat_interleave(Hq // Hkv, 1))
        ref = s.max(1) * D ** -0.5
        assert (np.abs(lse.double().cpu().numpy() - ref) <= np.abs(ref) * 6.1 * 2.0 ** -24).all()


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D", [(200, 333, 2, 1, 128), (700, 900, 2, 2, 64), (600, 1100, 2, 2, 128), (6, 500, 4, 1, 128), (4, 5000, 7, 1, 72)])
def test_ordinary_rows_beside_large_scores(ss, lq, lk, Hq, Hkv, D):
    """Every second token's scores are 2^40 times the others', in the same tiles. Tolerance of the others as in
    test_gpu_attn.py: scores to 4e-5 of their magnitudes, probabilities and outputs rounded by 2^-8."""
    g = torch.Generator(device="cuda").manual_seed(lk)
    q = torch.randn((lq, Hq, D), generator=g, device="cuda")
    q[0::2] *= 2.0 ** 40
    q = q.to(torch.bfloat16)
    k, v = (torch.randn((lk, Hkv, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    o = ss.attn(q, k, v).double().cpu().numpy()
    assert np.isfinite(o).all() and (np.abs(o) <= float(v.abs().max())).all()
    eo, _, mass, size = attention(*(t.float().cpu().numpy() for t in (q, k, v)), [0, lq], [0, lk])
    tol = mass * (2.0 ** -8 + size.T[:, :, None] * 8e-5 + 6e-5)
    tol = tol + 2.0 ** -8 * (np.abs(eo) + tol)
    assert (np.abs(o - eo) <= tol)[1::2].all()


def test_more_rows_than_a_join_can_hold(ss):
    """2^24 (token, head) rows over sequences long enough to be split: equal keys (stride 0), so the values come back."""
    B, Hq, Hkv, D, n = 65536, 256, 8, 8, 2048
    q = torch.randn((B, Hq, D), device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn((1, Hkv, D), device="cuda").to(torch.bfloat16).expand(B * n, Hkv, D) for _ in range(2))
    cq = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    o = ss.attn(q, k, v, cq, cq * n)
    assert torch.equal(o, v[:1].repeat_interleave(Hq // Hkv, 1).expand(B, Hq, D))
