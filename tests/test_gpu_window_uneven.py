"""attn under a window over contiguous sequences whose lengths are far from their mean, against the float64 oracle: a long one among
many of a few keys, first, last and between, with rows of its own or one token, and caches with room. Tolerances as in the tests
of the paged attention."""
import numpy as np
import pytest
import torch

from helpers import have_gpu
from test_gpu_window import _cum, _i32, _np, _run
from oracle.windowed import packed
from test_gpu_paged import compare

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 128), (6, 3, 64)])
@pytest.mark.parametrize("at", [0, 150, 299])
@pytest.mark.parametrize("lk,lq,window,sinks", [(9000, 1, 1 << 20, 0), (9000, 30, 1 << 20, 0), (9000, 30, 5000, 100), (9000, 1, 300, 4),
                                                (4000, 1, 1 << 20, 0), (700, 200, 600, 0)])
def test_one_long_sequence_among_short_ones(ss, Hq, Hkv, D, at, lk, lq, window, sinks):
    lens, rows = [(i * 5) % 9 for i in range(300)], [1] * 300
    lens[at], rows[at] = lk, lq
    q, k, v, o, lse = _run(ss, rows, lens, Hq, Hkv, D, window, sinks, seed=at)
    lse2 = torch.empty_like(lse)
    o2 = ss.attn(q, k, v, _i32(_cum(rows)), _i32(_cum(lens)), lse=lse2, window=window, sinks=sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_lengths_in_use_far_from_the_room(ss):
    B, room, Hkv, D, window = 40, 100, 2, 64, 1 << 20
    lens = [(i * 37) % 101 for i in range(B)]
    ck = [b * room for b in range(B)] + [B * room + 6000]  # the last one has the rest of the cache
    lens[-1] = 5001
    q = torch.randn((B, 4, D), device="cuda").to(torch.bfloat16)
    k, v = (torch.full((ck[-1], Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for b, n in enumerate(lens):
        for t in (k, v):
            t[ck[b] : ck[b] + n] = torch.randn((n, Hkv, D), device="cuda").to(torch.bfloat16)
    o = ss.attn(q, k, v, _i32(list(range(B + 1))), _i32(ck), k_len=_i32(lens), window=window)
    compare(o, None, packed(_np(q), np.nan_to_num(_np(k)), np.nan_to_num(_np(v)), list(range(B + 1)), ck, lens, True, window, 0))
