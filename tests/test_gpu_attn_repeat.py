"""attn gives the same bits in every call: thousands of calls in a row of each form of its kernels (few rows whole and in parts,
tiles of many rows, keys in two parts, windows over caches and prompts), with sequences that end inside a unit of keys, so that loads
to LDS of very different latency are in flight beside the reads of the unit before."""
import numpy as np
import pytest
import torch

from helpers import have_gpu
from oracle.windowed import packed
from test_gpu_paged import compare

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

CALLS = 3000
CASES = {  # rows, keys, query heads, key heads, window, sinks
    "chunks in parts": ([29, 13], [1000, 777], 16, 2, 0, 0),
    "one token in parts": ([1], [3999], 32, 8, 0, 0),
    "tokens, whole and short": ([1] * 9, [5, 33, 0, 64, 77, 300, 1, 31, 200], 8, 2, 0, 0),
    "tokens in a few parts": ([1] * 40, [1100 + 13 * i for i in range(40)], 8, 2, 0, 0),
    "prompts": ([129, 50], [1000, 777], 64, 2, 0, 0),
    "a prompt in two parts": ([300], [1333], 2, 1, 0, 0),
    "window, chunks": ([29, 13], [1000, 777], 16, 2, 300, 5),
    "window, tokens": ([1] * 9, [5, 33, 0, 64, 77, 3000, 1, 31, 2000], 8, 2, 1000, 4),
    "window, prompts": ([300, 150], [333, 177], 6, 2, 100, 3),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("D", [64, 128])
def test_many_calls_give_the_same_bits(name, D):
    import structured_sparse_quantized_amd as ss
    lq, lk, Hq, Hkv, window, sinks = CASES[name]
    g = torch.Generator(device="cuda").manual_seed(D)
    q = torch.randn((sum(lq), Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((sum(lk), Hkv, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cq, ck = (np.concatenate([[0], np.cumsum(n)]).astype(int).tolist() for n in (lq, lk))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cu_q, cu_k = i32(cq), i32(ck)
    lse, lse0 = (torch.empty((Hq, sum(lq)), device="cuda") for _ in range(2))
    call = lambda l, out=None: ss.attn(q, k, v, cu_q, cu_k, lse=l, out=out, window=window or None, sinks=sinks)  # noqa: E731
    first = call(lse0).clone()
    np64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    compare(first, lse0, packed(np64(q), np64(k), np64(v), cq, ck, None, True, window, sinks))
    out, wrong = torch.empty_like(first), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(CALLS):
        call(lse, out)
        wrong += (out != first).any() | (lse != lse0).any()
    assert int(wrong) == 0
