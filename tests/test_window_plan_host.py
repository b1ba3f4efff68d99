"""How calls of few rows a sequence under a window are cut (no GPU needed): the kernel sums the units of all tiles in 31 bits, so
a call whose sum could pass them has to leave its tiles whole, which asks for no workspace."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "structured_sparse_quantized_amd", "libss.so")),
                                reason="libss.so not built")


def units(seqs, Hq, Hkv, window, sinks):
    """Units of 32 keys of all tiles of 32 rows of a key head; seqs: (how many, query rows, keys) of each kind of sequence."""
    G, total = Hq // Hkv, 0
    for n, lq, lk in seqs:
        tokens = min((32 + G - 2) // G + 1, lq)
        seen = (window + tokens - 1 + 62) // 32 + (sinks + 31) // 32
        total += n * -(-lq * G // 32) * Hkv * max(min(-(-lk // 32), seen), 1)
    return total


# mostly one sequence with nearly all rows and keys: the mean length says little about the sum
SKEWED = [([(2047, 0, 0), (1, 16384, 1 << 22)], 32, 8, 128, 1 << 22, 0),
          ([(4095, 1, 1), (1, 126000, 560000)], 32, 32, 8, 1 << 30, 0),
          ([(4095, 1, 1), (1, 126000, 560000)], 32, 32, 8, 300000, 250000),
          ([(1023, 1, 30), (1, 30000, 3000000)], 64, 64, 8, 1 << 30, 4),
          ([(300, 3, 50), (1, 8000, 4500000)], 64, 64, 8, 1 << 30, 0)]


@pytest.mark.parametrize("seqs,Hq,Hkv,D,window,sinks", SKEWED, ids=lambda v: str(v)[:40])
def test_sums_beyond_31_bits_are_not_cut(seqs, Hq, Hkv, D, window, sinks):
    import structured_sparse_quantized_amd as ss
    B, Tq, Tk = (sum(n * x for n, x in zip([s[0] for s in seqs], col)) for col in zip(*[(1, s[1], s[2]) for s in seqs]))
    assert units(seqs, Hq, Hkv, window, sinks) >= 1 << 31
    assert ss.attn_window_workspace_bytes(Tq, Tk, B, Hq, Hkv, D, window, sinks) == 0


def test_sums_within_31_bits_are_cut():
    import structured_sparse_quantized_amd as ss
    assert units([(64, 1, 8192)], 32, 8, 4096, 4) < 1 << 31
    assert ss.attn_window_workspace_bytes(64, 64 * 8192, 64, 32, 8, 128, 4096, 4) > 0
    assert ss.attn_window_workspace_bytes(64, 64 * 8192, 64, 32, 8, 128, 1 << 30, 4) > 0


def test_short_sequences_are_cut_where_one_of_them_may_be_long():
    """A tile stays whole, without a workspace, where the mean is at most 128 keys and no sequence can have more than 4096."""
    import structured_sparse_quantized_amd as ss
    need = lambda B, Tk, window, sinks=0: ss.attn_window_workspace_bytes(B, Tk, B, 32, 8, 128, window, sinks)  # noqa: E731
    assert need(1024, 1023 * 8 + 100000, 1 << 20) > 0 and need(81, 80 * 8 + 8000, 9000) > 0
    assert need(64, 64 * 60, 1 << 20) == 0 and need(1, 128, 4096) == 0 and need(16, 16 * 128, 4096) == 0
    assert need(1024, 1023 * 8 + 100000, 3000, 4) == 0  # the window keeps tiles short, whatever the lengths
    assert need(64, 64 * 200, 1 << 20) > 0
