"""attn under a window in calls so long that the units of all tiles pass 31 bits: one sequence with nearly all rows and keys among
thousands of a single key (tests/test_window_plan_host.py counts them). Every row is written, and a sample of them is compared
with float64.

Tolerances: those of tests/test_gpu_paged.py, and what a float32 sum of 560000 positive powers may lose on its way: a lane adds 16
of 32 keys to its sum at a time, every second unit, 8750 times, each rounding 2^-24 of the sum at most; the product's sums
take 17500 steps of 32 keys, two of 16 each, over half of them: 17500 roundings."""
import pytest
import torch

from helpers import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

SHORT, ROWS, KEYS, H, D = 4095, 126000, 560000, 32, 8


@pytest.mark.parametrize("window,sinks", [(1 << 30, 0), (300000, 250000)])
def test_a_long_sequence_among_thousands_of_one_key(window, sinks):
    import structured_sparse_quantized_amd as ss
    g = torch.Generator(device="cuda").manual_seed(1)
    Tq, Tk, at = SHORT + ROWS, SHORT + KEYS, 2000  # the long one is sequence `at`
    q = torch.randn((Tq, H, D), generator=g, device="cuda").to(torch.bfloat16)
    # keys and values of a head adjacent; values around 1, so that a row's result is not what roundings leave of zero
    k = torch.randn((H, Tk, D), generator=g, device="cuda").to(torch.bfloat16)
    v = (1 + torch.randn((H, Tk, D), generator=g, device="cuda") / 2).to(torch.bfloat16)
    cu_q = torch.tensor(list(range(at + 1)) + [at + ROWS + i for i in range(SHORT - at + 1)], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor(list(range(at + 1)) + [at + KEYS + i for i in range(SHORT - at + 1)], dtype=torch.int32, device="cuda")
    assert cu_q.numel() == SHORT + 2 and int(cu_q[-1]) == Tq and int(cu_k[-1]) == Tk
    o = torch.full((Tq, H, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    lse = torch.full((H, Tq), float("nan"), device="cuda")
    ss.attn(q, k.transpose(0, 1), v.transpose(0, 1), cu_q, cu_k, out=o, lse=lse, window=window, sinks=sinks)
    assert not o.isnan().any() and not lse.isnan().any()
    # a sequence of one key: its value
    for rows, keys in ((slice(0, at), slice(0, at)), (slice(at + ROWS, Tq), slice(at + KEYS, Tk))):
        assert torch.equal(o[rows], v[:, keys].transpose(0, 1))
    for r in (0, 1, 40000, 77777, ROWS - 1):
        p = r + KEYS - ROWS
        j = torch.arange(p + 1, device="cuda")
        j = at + j[(j > p - window) | (j < sinks)]
        qd, kd, vd = q[at + r].double(), k[:, j].double(), v[:, j].double()
        s = (kd * qd[:, None]).sum(-1) * D ** -0.5
        size = (kd * qd[:, None]).abs().sum(-1).amax(1, keepdim=True) * D ** -0.5
        el = torch.logsumexp(s, 1, keepdim=True)
        e = torch.exp(s - el)[..., None]
        eo, mass = (e * vd).sum(1), (e * vd.abs()).sum(1)
        adds = 26250 * 2.0 ** -24
        tol = mass * (2.0 ** -8 + 8e-5 * size + 6e-5 + adds)
        tol = tol + 2.0 ** -8 * (eo.abs() + tol)
        err = (o[at + r].double() - eo).abs()
        assert (err <= tol).all(), (r, (err / tol).max())
        assert err.norm() <= (2.0 ** -8 + adds) * eo.norm()
        lerr = (lse[:, at + r].double() - el[:, 0]).abs()
        assert (lerr <= size[:, 0] * 4e-5 + 2e-5 + el[:, 0].abs() * 2.0 ** -22 + 8750 * 2.0 ** -24).all(), (r, lerr.max())
