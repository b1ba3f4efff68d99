"""attn with a sliding window and first tokens that stay visible, against the float64 oracle: packed prompts in every form of
the kernels (tiles of many rows, keys in two parts, few rows), contiguous caches with room, windows from one key to more than
there are. Tolerances as in the tests of the paged attention."""
import numpy as np
import pytest
import torch

from helpers import have_gpu
from oracle.windowed import packed
from test_gpu_paged import compare

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(int).tolist()


def _np(t):
    return t.double().cpu().numpy()


def _run(ss, lq, lk, Hq, Hkv, D, window, sinks, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((sum(lq), Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((sum(lk), Hkv, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    lse = torch.full((Hq, sum(lq)), 7.0, device="cuda")
    cq, ck = _cum(lq), _cum(lk)
    o = ss.attn(q, k, v, _i32(cq), _i32(ck), lse=lse, window=window, sinks=sinks)
    compare(o, lse, packed(_np(q), _np(k), _np(v), cq, ck, None, True, window, sinks))
    return q, k, v, o, lse


WINDOWS = [(1, 0), (1, 2), (5, 0), (31, 1), (32, 0), (33, 33), (63, 0), (64, 64), (65, 4), (127, 100), (128, 0), (200, 300),
           (1000, 1), (100000, 5)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("lq,lk", [([300], [300]), ([200], [450]), ([150, 1, 0, 97], [150, 60, 5, 20]), ([5, 3], [700, 2])], ids=str)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 128), (3, 3, 64), (7, 1, 72)])
def test_packed(ss, window, sinks, lq, lk, Hq, Hkv, D):
    _run(ss, lq, lk, Hq, Hkv, D, window, sinks, seed=window)


@pytest.mark.parametrize("window,sinks", [(700, 0), (1500, 70), (1100, 4)])
@pytest.mark.parametrize("lq,lk,Hq,Hkv,D", [([1300], [1300], 2, 2, 64), ([1700], [1700], 2, 1, 128), ([600], [2500], 4, 4, 64)])
def test_keys_in_two_parts(ss, window, sinks, lq, lk, Hq, Hkv, D):
    _run(ss, lq, lk, Hq, Hkv, D, window, sinks)


@pytest.mark.parametrize("D", [8, 16, 40, 56, 64, 80, 96, 120, 128])
def test_head_sizes(ss, D):
    _run(ss, [140, 33], [140, 50], 4, 2, D, 40, 3, seed=D)


@pytest.mark.parametrize("G", [32, 40, 64])
def test_a_token_a_tile(ss, G):
    _run(ss, [20], [75], G, 1, 64, 10, 2)
    _run(ss, [2], [500], G, 1, 128, 100, 2)


def test_a_window_that_hides_nothing_is_no_window(ss):
    q, k, v, o, lse = _run(ss, [200, 90], [260, 90], 4, 2, 128, 100000, 0)
    assert torch.equal(o, ss.attn(q, k, v, _i32([0, 200, 290]), _i32([0, 260, 350])))


@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 3), (100, 0), (1000, 4), (5000, 0)])
@pytest.mark.parametrize("lens,room", [([0, 5, 900, 1], 1000), ([6000], 8000), ([40] * 70, 64)], ids=lambda v: str(v)[:20])
def test_caches_with_room(ss, window, sinks, lens, room):
    """NaN behind the keys in use, and before the windows."""
    B, Hkv, D = len(lens), 2, 64
    q = torch.randn((B, 6, D), device="cuda").to(torch.bfloat16)
    k, v = (torch.full((B * room, Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for b, n in enumerate(lens):
        low = max(n - window, 0)
        for t in (k, v):
            for a, e in ((0, min(sinks, n)), (low, n)):
                t[b * room + a : b * room + e] = torch.randn((e - a, Hkv, D), device="cuda").to(torch.bfloat16)
    ck = [b * room for b in range(B + 1)]
    o = ss.attn(q, k, v, _i32(list(range(B + 1))), _i32(ck), k_len=_i32(lens), window=window, sinks=sinks)
    compare(o, None, packed(_np(q), np.nan_to_num(_np(k)), np.nan_to_num(_np(v)), list(range(B + 1)), ck, lens, True, window, sinks))


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D,window,sinks", [
    (90, 200, 3, 1, 64, 50, 4), (200, 333, 2, 1, 128, 64, 0), (700, 1700, 2, 2, 64, 600, 3), (6, 500, 4, 1, 128, 30, 2),
    (20, 75, 40, 1, 64, 10, 2)])
def test_infinities_and_nan_reach_the_rows_that_see_them(ss, lq, lk, Hq, Hkv, D, window, sinks):
    q, k, v, clean, lse = _run(ss, [lq], [lk], Hq, Hkv, D, window, sinks)
    p = torch.arange(lq, device="cuda") + lk - lq
    for j in sorted({0, 1, sinks, 7, lk - 1, lk - 2, lk - lq, max(lk - lq - 5, 0), max(lk - window, 0), max(lk - window - 3, 0), lk // 2}):
        rows = (p >= j) & ((p - window < j) | (j < sinks))
        vb = v.clone()
        vb[j, :, 1], vb[j, :, 3] = float("nan"), float("inf")
        o = ss.attn(q, k, vb, window=window, sinks=sinks)
        assert torch.equal(o[~rows], clean[~rows])
        other = [c for c in range(D) if c not in (1, 3)]
        assert torch.equal(o[:, :, other], clean[:, :, other])
        assert o[rows][:, :, 1].isnan().all() and (o[rows][:, :, 3] == float("inf")).all()
        kb = k.clone()
        kb[j, :, 2] = float("nan")
        o = ss.attn(q, kb, v, window=window, sinks=sinks)
        assert torch.equal(o[~rows], clean[~rows]) and o[rows].isnan().all()


def test_captured_and_replayed(ss):
    q = torch.zeros((3, 8, 64), device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn((3 * 4000, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    cu, ck, n = _i32([0, 1, 2, 3]), _i32([0, 4000, 8000, 12000]), _i32([1, 1, 1])
    call = lambda: ss.attn(q, k, v, cu, ck, k_len=n, window=1000, sinks=4)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for lens in ([1, 4000, 0], [3999, 17, 1000], [2000, 2001, 2002]):
        n.copy_(_i32(lens))
        q.copy_(torch.randn(q.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        first = got.clone()
        assert torch.equal(first, call())
        compare(first, None, packed(_np(q), _np(k), _np(v), [0, 1, 2, 3], [0, 4000, 8000, 12000], lens, True, 1000, 4))
