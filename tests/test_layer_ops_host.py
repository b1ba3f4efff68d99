"""Host side of the calls between products (no GPU needed): plans of large batches, the
package without its binding."""
import os
import subprocess
import sys

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


@built
def test_the_package_imports_without_its_binding():
    """_ssbind serves the calls between products alone: where it does not load (another Python or torch), everything else
    works as before, and those calls say what is missing."""
    code = """
import sys
sys.modules["structured_sparse_quantized_amd._ssbind"] = None  # (makes its import fail)
import torch
import structured_sparse_quantized_amd as ss
assert ss.lifted_k(100, 2) == 256 and ss.rotary_steps(8, device="cpu")[0].shape == (4,)
assert ss.attn_workspace_bytes(1, 9000, 1, 8, 2, 64) > 0
t = torch.zeros((4, 2, 16), dtype=torch.bfloat16)
for call in (lambda: ss.attn(t, t, t), lambda: ss.rotary(t, t, t), lambda: ss.spgemm_tiled_epilogue(0, 1, 1, 256, t, t, t)):
    try:
        call()
    except ImportError as e:
        assert "_ssbind" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("no ImportError")
try:
    ss.quant_lift_act(t[0].float(), 2, "i8")
except ss.SSError as e:
    print("served:", e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "served" in r.stdout, r.stderr
