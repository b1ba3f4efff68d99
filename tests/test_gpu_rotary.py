"""ss_rotary on the GPU against the float64 oracle: layouts, part of the head, scalings, far positions, strides,
in place, inverse, sizes that vectors do not divide, another stream, a captured graph.

Tolerance. An angle is off by at most 2^-25 half turns (its rounding to float32) + 2^-31, times pi; sin and cos by
2 units in the last place; the factor mscale, the product and the fused multiply-add round once each: together
less than 2^-21 of mscale (|a| + |b|). bf16 outputs round by at most 2^-8 of the value, float32 ones by 2^-24."""
import numpy as np
import pytest
import torch

from helpers import have_gpu
from oracle.rotary import frequencies, rotary

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


def _check(got, x, pos, f, layout, m, inverse=False):
    xd = x.double().cpu().numpy()
    exp = rotary(xd, pos.cpu().numpy(), f, layout, m, inverse)
    n = len(f)
    size = np.zeros_like(xd)
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    size[..., a] = size[..., b] = np.abs(xd[..., a]) + np.abs(xd[..., b])
    tol = 2.0 ** -21 * m * size
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    tol = tol + half * (np.abs(exp) + tol)
    g = got.double().cpu().numpy()
    assert (np.abs(g - exp) <= tol)[..., : 2 * n].all(), float((np.abs(g - exp) / (tol + 1e-300)).max())
    assert np.array_equal(g[..., 2 * n :], xd[..., 2 * n :])


CASES = [  # T, H, D, rot
    (1, 1, 2, 2), (1, 40, 128, 128), (5, 3, 64, 32), (7, 2, 80, 80), (3, 5, 100, 74), (130, 14, 96, 64), (2, 1, 256, 254),
    (33, 9, 128, 16), (600, 40, 128, 128)]


@pytest.mark.parametrize("T,H,D,rot", CASES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rotary(ss, T, H, D, rot, layout, dt):
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + D)
    x = torch.randn((T, H, D), generator=g, device="cuda").to(dt)
    pos = torch.randint(-5, 2000000, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    steps, m = ss.rotary_steps(rot)
    f, _ = frequencies(rot)
    y = ss.rotary(x, pos, steps, layout)
    _check(y, x, pos, f, layout, 1.0)
    z = x.clone()
    assert ss.rotary(z, pos, steps, layout, out=z) is z and torch.equal(z, y)  # in place
    _check(ss.rotary(x, pos, steps, layout, inverse=True), x, pos, f, layout, 1.0, True)


@pytest.mark.parametrize("plan", [dict(base=500000.0, scaling="smooth", factor=8.0, original=8192, high=4.0),
                                  dict(scaling="yarn", factor=4.0, original=4096, high=32.0), dict(scaling="ntk", factor=2.0),
                                  dict(scaling="linear", factor=3.0)], ids=lambda p: p["scaling"])
def test_scalings_on_strided_heads(ss, plan):
    """The query and key heads inside a projection's output, written to another strided place."""
    T, Hq, Hkv, D = 65, 7, 2, 64
    row = torch.randn((T, (Hq + 2 * Hkv) * D + 8), device="cuda").to(torch.bfloat16)
    x = row[:, 8:].unflatten(1, (Hq + 2 * Hkv, D))[:, : Hq + Hkv]
    dst = torch.full((Hq + Hkv, T + 3, D + 8), 7.0, device="cuda", dtype=torch.bfloat16)
    out = dst[:, :T, :D].transpose(0, 1)  # head-major
    pos = torch.arange(100000, 100000 + T, device="cuda", dtype=torch.int32)
    steps, m = ss.rotary_steps(D, **plan)
    f, om = frequencies(D, **plan)
    assert ss.rotary(x, pos, steps, mscale=m, out=out) is out
    _check(out, x, pos, f, "half", om)
    assert (dst[:, T:] == 7).all() and (dst[:, :, D:] == 7).all()
    before = row.clone()
    ss.rotary(x, pos, steps, mscale=m, out=x)  # in place inside the row: the rest of it stays
    assert torch.equal(x, out) and torch.equal(row[:, :8], before[:, :8])
    assert torch.equal(row[:, 8 + (Hq + Hkv) * D :], before[:, 8 + (Hq + Hkv) * D :])


def test_unaligned_views(ss):
    """Views that start between vectors, and odd strides, take the element path."""
    base = torch.randn(1 + 9 * 5 * 67, device="cuda").to(torch.bfloat16)
    x = base[1:].view(9, 5, 67)[:, :, :64]
    pos = torch.arange(9, device="cuda", dtype=torch.int32) * 1001
    steps, _ = ss.rotary_steps(64)
    f, _ = frequencies(64)
    for layout in ("half", "interleaved"):
        _check(ss.rotary(x, pos, steps, layout), x, pos, f, layout, 1.0)


def test_gradient(ss):
    """The turn is linear: its gradient is the inverse turn times mscale, and differences agree."""
    x, w = torch.randn((6, 2, 32), device="cuda"), torch.randn((6, 2, 32), device="cuda")
    pos = torch.arange(6, device="cuda", dtype=torch.int32) + 50
    steps, m = ss.rotary_steps(16, scaling="yarn", factor=4.0, original=64, high=8.0)
    grad = ss.rotary(w, pos, steps, mscale=m, inverse=True)  # of sum(w * rotary(x)) in x
    f, om = frequencies(16, scaling="yarn", factor=4.0, original=64, high=8.0)
    _check(grad, w, pos, f, "half", om, True)
    xd, wd = x.double().cpu().numpy(), w.double().cpu().numpy()
    for at in ((0, 0, 0), (3, 1, 9), (5, 0, 20)):
        d = np.zeros_like(xd)
        d[at] = 0.5  # exact for a linear map
        diff = (wd * (rotary(xd + d, pos.cpu().numpy(), f, "half", om) - rotary(xd - d, pos.cpu().numpy(), f, "half", om))).sum()
        assert abs(diff - float(grad[at])) <= 2.0 ** -19 * om * (abs(wd).max() * 2)


def test_stream_and_graph(ss):
    x = torch.randn((64, 8, 128), device="cuda").to(torch.bfloat16)
    pos = torch.arange(64, device="cuda", dtype=torch.int32)
    steps, _ = ss.rotary_steps(128)
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ss.rotary(x, pos, steps, out=y)
    s.synchronize()
    assert torch.equal(y, ss.rotary(x, pos, steps))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.rotary(x, pos, steps, out=y)
    for k in range(3):
        x.copy_(torch.randn((64, 8, 128), device="cuda"))
        pos.add_(1000 * k)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ss.rotary(x, pos, steps))


def test_offsets_beyond_32_bits(ss):
    T, H, D = 430000, 40, 128
    steps, m = ss.rotary_steps(D)
    x = torch.zeros((T, H, D), device="cuda", dtype=torch.bfloat16)
    x[-50:] = torch.randn((50, H, D), device="cuda").to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    want = ss.rotary(x[-50:].clone(), pos[-50:].clone(), steps, mscale=m)
    assert torch.equal(ss.rotary(x, pos, steps, mscale=m)[-50:], want)
    assert torch.equal(ss.rotary(x, pos, steps, mscale=m, out=x)[-50:], want)


def test_empty_and_refused(ss):
    steps, _ = ss.rotary_steps(32)
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert ss.rotary(torch.empty((0, 3, 32), device="cuda"), pos, steps).shape == (0, 3, 32)
    x = torch.zeros((4, 3, 32), device="cuda")
    p = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: ss.rotary(x, p.long(), steps), lambda: ss.rotary(x, p[:3], steps),
                lambda: ss.rotary(x[:, :, ::2], p, steps), lambda: ss.rotary(x, p.cpu(), steps),
                lambda: ss.rotary(x, p, steps.int()), lambda: ss.rotary(x[..., :16], p, steps),
                lambda: ss.rotary(x, p, steps, out=x.bfloat16()), lambda: ss.rotary(x, p, steps, "other"),
                lambda: ss.rotary(x, p, steps, out=torch.zeros(1, 3, 32, device="cuda").expand(4, 3, 32))):
        with pytest.raises(ss.SSError):
            bad()
