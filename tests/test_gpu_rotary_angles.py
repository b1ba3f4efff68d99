"""ss_rotary's angles next to the quarter turns, where sin or cos is small, relative to their values."""
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


@pytest.mark.parametrize("quarter", [0, 1, 2, 3])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_angles_next_to_a_quarter_turn(ss, quarter, layout):
    """Steps of quarter / 4 turns and a little, at position 1 (and of the opposite sign at -1): (1, 0) turns to (cos, sin).
    The little is a multiple of 2^-34 turns, kept exactly as an integer; it rounds to float32 by 2^-24, sin and cos are good to
    4 units in the last place, 2^-21 of the value, and nothing else rounds."""
    little = np.array([s * k << 30 for k in (1, 2, 3, 5, 40, 63, 129, 1000, 77777, 10 ** 7, 10 ** 8) for s in (1, -1)], dtype=np.int64)
    words = ((quarter << 62) + little.astype(object)) % (1 << 64)
    steps = torch.from_numpy(np.array(words, dtype=np.uint64).view(np.int64)).cuda()
    n = len(little)
    x = torch.zeros((2, 1, 2 * n), device="cuda")
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    x[:, :, a] = 1.0
    pos = torch.tensor([1, -1], dtype=torch.int32, device="cuda")
    y = ss.rotary(x, pos, steps, layout).double().cpu().numpy()[:, 0]
    for row, sign in ((0, 1), (1, -1)):
        q = sign * quarter % 4
        t = [sign * int(v) * math.pi * 2.0 ** -63 for v in little]
        cos, sin = [math.cos(v) for v in t], [math.sin(v) for v in t]
        for _ in range(q):  # a quarter turn on
            cos, sin = [-v for v in sin], cos
        for got, want in ((y[row, a], np.array(cos)), (y[row, b], np.array(sin))):
            assert (np.abs(got - want) <= (2.0 ** -24 + 2.0 ** -21) * 1.01 * np.abs(want)).all(), (got / want - 1)
