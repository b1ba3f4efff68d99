"""Host side of the calls between products (no GPU needed): plans of large batches."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "structured_sparse_quantized_amd", "libss.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="libss.so not built")


@built
def test_attention_parts_stay_within_a_launch():
    """Joining the parts takes 256 threads a row (token, head): from 2^24 rows on a launch cannot hold them, and the keys
    are not split."""
    import structured_sparse_quantized_amd as ss
    for B, Hq in ((65536, 256), (1 << 18, 64), (1 << 19, 32)):
        assert ss.attn_workspace_bytes(B, 2048 * B, B, Hq, 8, 8) == 0
        assert ss.attn_workspace_bytes(B - 1, 2048 * (B - 1), B - 1, Hq, 8, 8) > 0
