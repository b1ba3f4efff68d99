"""Pins of the rotary and attention oracles, and the host side of the two calls (no GPU needed): frequencies,
refusals, empty calls."""
import ctypes
import math
import os

import numpy as np
import pytest

from oracle.attention import attention
from oracle.rotary import frequencies, rotary

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "structured_sparse_quantized_amd", "libss.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="libss.so not built")

PLANS = [dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
         dict(base=500000.0, scaling="smooth", factor=8.0, original=8192, low=1.0, high=4.0),
         dict(scaling="yarn", factor=4.0, original=4096, low=1.0, high=32.0)]


def test_rotary_is_a_rotation_of_positions():
    rng = np.random.default_rng(0)
    f, _ = frequencies(16)
    assert f[0] == 1.0 and np.isclose(f[-1], 10000.0 ** (-14 / 16))
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    for layout in ("half", "interleaved"):
        dot = [float((rotary(q, [p], f, layout) * rotary(k, [p - 7], f, layout)).sum()) for p in (7, 100, 12345)]
        assert np.allclose(dot, dot[0], atol=1e-9)  # only the distance counts
        back = rotary(rotary(q, [99], f, layout), [99], f, layout, inverse=True)
        assert np.allclose(back, q, atol=1e-12)
    x = np.zeros((1, 1, 4))
    x[0, 0, 0] = 1
    y = rotary(x, [1], [math.pi / 2, 0.0], "half")
    assert np.allclose(y[0, 0], [0, 0, 1, 0])  # value 0 pairs with value 2
    y = rotary(x, [1], [math.pi / 2, 0.0], "interleaved")
    assert np.allclose(y[0, 0], [0, 1, 0, 0])  # with value 1


def test_scalings_at_their_ends():
    plain, _ = frequencies(128, 500000.0)
    smooth, m = frequencies(128, 500000.0, "smooth", 8.0, 8192, 1.0, 4.0)
    turns = 8192 * plain / (2 * math.pi)
    assert m == 1.0 and np.allclose(smooth[turns >= 4], plain[turns >= 4]) and np.allclose(smooth[turns <= 1], plain[turns <= 1] / 8)
    assert (smooth <= plain).all() and (smooth >= plain / 8).all()
    yarn, m = frequencies(64, 10000.0, "yarn", 4.0, 4096, 1.0, 32.0)
    plain, _ = frequencies(64)
    assert np.isclose(m, 1.1386294361) and yarn[0] == plain[0] and np.isclose(yarn[-1], plain[-1] / 4)
    ntk, _ = frequencies(64, 10000.0, "ntk", 4.0)
    assert np.isclose(ntk[-1], plain[-1] / 4) and ntk[0] == 1.0  # the slowest pair is stretched by the factor


def test_attention_by_hand():
    q = np.zeros((2, 2, 2))
    k = np.zeros((3, 1, 2))
    v = np.arange(6, dtype=float).reshape(3, 1, 2)
    o, lse, _, _ = attention(q, k, v, [0, 2], [0, 3])
    assert np.allclose(o[0, 0], v[:2, 0].mean(0)) and np.allclose(o[1, 1], v[:, 0].mean(0))
    assert np.allclose(lse[:, 0], math.log(2)) and np.allclose(lse[:, 1], math.log(3))
    o, lse, _, _ = attention(q, k, v, [0, 2], [0, 3], k_len=[1])  # more rows than keys: the first sees none
    assert (o[0] == 0).all() and np.isneginf(lse[:, 0]).all() and np.allclose(o[1, 0], v[0, 0])
    o, _, _, _ = attention(q, k, v, [0, 1, 2], [0, 1, 3], causal=False)
    assert np.allclose(o[0, 0], v[0, 0]) and np.allclose(o[1, 0], v[1:, 0].mean(0))


@built
@pytest.mark.parametrize("plan", PLANS, ids=lambda p: p.get("scaling", "none") + str(p.get("base", "")))
@pytest.mark.parametrize("rot", [2, 20, 64, 128])
def test_steps_match_the_oracle(plan, rot):
    import structured_sparse_quantized_amd as ss
    steps, m = ss.rotary_steps(rot, device="cpu", **plan)
    f, om = frequencies(rot, **plan)
    got = steps.numpy().view(np.uint64).astype(np.float64) * 2.0 ** -64 * 2 * math.pi
    # the oracle's own rounding: pow and the few operations after it, 2^-52 each; a step is a whole number of
    # 2^-64 turns, so it is off by up to half of that, 2 pi 2^-65 radians, whatever the frequency's size
    assert steps.shape == (rot // 2,) and np.isclose(m, om, rtol=2.0 ** -23)
    assert np.allclose(got, f, rtol=64 * 2.0 ** -52, atol=2 * math.pi * 2.0 ** -65)


FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first


@built
def test_rotary_refusals():
    import structured_sparse_quantized_amd as ss
    L = ss.lib
    buf, m = (ctypes.c_int64 * 8)(), ctypes.c_float()

    def steps(rot=8, base=1e4, sc=0, factor=1.0, orig=0.0, low=1.0, high=4.0, out=buf):
        return L.ss_rotary_steps(rot, base, sc, factor, orig, low, high, out, ctypes.byref(m))

    assert steps() == ss.SS_OK
    assert steps(rot=7) == steps(rot=0) == steps(base=0.0) == steps(base=float("nan")) == steps(factor=-1.0) == ss.SS_ERR_SHAPE
    assert steps(sc=3) == steps(sc=4, orig=100.0, low=4.0) == steps(sc=4, orig=100.0, base=1.0) == ss.SS_ERR_SHAPE
    assert steps(sc=5) == ss.SS_ERR_UNSUPPORTED and steps(out=None) == ss.SS_ERR_NULL

    def call(x=FAKE, dt=ss.SS_BF16, T=4, H=2, D=16, sxt=32, sxh=16, pos=FAKE, st=FAKE, rot=16, lay=0, ms=1.0, y=FAKE,
             syt=32, syh=16):
        return L.ss_rotary(x, dt, T, H, D, sxt, sxh, pos, st, rot, lay, ms, 0, y, syt, syh, None)

    assert call(dt=ss.SS_I8) == ss.SS_ERR_DTYPE
    assert call(T=-1) == call(rot=15) == call(rot=18) == call(rot=0) == call(sxt=-8) == call(syh=8) == ss.SS_ERR_SHAPE
    assert call(x=None) == call(pos=None) == call(st=None) == call(y=None) == ss.SS_ERR_NULL
    assert call(sxt=64) == ss.SS_ERR_SHAPE  # in place with other strides
    assert call(lay=2) == ss.SS_ERR_UNSUPPORTED and call(ms=float("inf")) == ss.SS_ERR_SHAPE
    assert call(x=ctypes.c_void_p((1 << 20) + 1)) == ss.SS_ERR_ALIGN
    assert call(T=0, x=None) == call(H=0, x=None) == ss.SS_OK
    with pytest.raises(ss.SSError):
        ss.rotary_steps(64, scaling="cubic", device="cpu")


@built
def test_attention_refusals():
    import torch
    import structured_sparse_quantized_amd as ss
    odd = ctypes.c_void_p((1 << 20) + 8)

    def call(q=FAKE, st=64, sh=16, k=FAKE, skt=64, skh=16, o=FAKE, sot=64, Tq=8, Tk=8, B=1, Hq=4, Hkv=2, D=16, cq=FAKE,
             ck=FAKE, scale=0.25, ws=FAKE, n=1 << 40, lse=None):
        return ss.lib.ss_attn(q, st, sh, k, skt, skh, k, skt, skh, o, sot, 16, lse, Tq, Tk, B, Hq, Hkv, D, cq, ck, None,
                              scale, 1, ws, n, None)

    assert call(Tq=-1) == call(Hq=3) == call(Hkv=0) == call(n=-1) == ss.SS_ERR_SHAPE
    assert call(scale=0.0) == call(scale=-1.0) == call(scale=float("nan")) == call(scale=float("inf")) == ss.SS_ERR_SHAPE
    assert call(D=20) == call(D=136) == call(D=4) == ss.SS_ERR_UNSUPPORTED
    assert call(q=None) == call(k=None) == call(o=None) == ss.SS_ERR_NULL
    assert call(q=odd) == call(k=odd) == call(o=odd) == call(st=60) == call(skh=12) == call(lse=ctypes.c_void_p(2)) == ss.SS_ERR_ALIGN
    assert call(sot=8) == call(st=-64) == ss.SS_ERR_SHAPE
    assert call(skt=1 << 24) == ss.SS_ERR_UNSUPPORTED
    assert call(B=1 << 27, Hq=64, Hkv=64) == call(Tq=1 << 30, Hq=512, Hkv=512) == ss.SS_ERR_SHAPE  # 2^32 threads and more
    assert call(B=2, cq=None) == call(B=2, ck=None) == ss.SS_ERR_NULL
    assert call(Tq=0, q=None) == call(B=0) == call(Hq=0, Hkv=0) == ss.SS_OK
    need = ss.attn_workspace_bytes(8, 10000, 1, 4, 2, 16)  # few rows, many keys: split over workgroups
    few = dict(Tk=10000)
    assert need > 0 and need % (8 * 4 * 17 * 4) == 0
    assert call(ws=None, **few) == ss.SS_ERR_NULL and call(n=need - 1, **few) == ss.SS_ERR_SHAPE and call(ws=odd, **few) == ss.SS_ERR_ALIGN
    assert ss.attn_workspace_bytes(8000, 8000, 1, 4, 2, 16) == 0
    assert ss.lib.ss_attn_workspace_bytes(8, 8, 1, 3, 2, 16) == -1 and ss.attn_workspace_bytes(0, 8, 1, 4, 2, 16) == 0
    t = torch.zeros((4, 2, 16), dtype=torch.bfloat16)
    for bad in (lambda: ss.attn(t, t, t), lambda: ss.attn(t.float(), t, t), lambda: ss.attn(t[0], t, t),
                lambda: ss.attn(t, t[:, :, :8], t), lambda: ss.attn(t, t, t, lse=torch.zeros(2, 3)),
                lambda: ss.rotary(t, torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int64)),
                lambda: ss.rotary(t, torch.zeros(4), torch.zeros(8)), lambda: ss.rotary(t.half(), None, None)):
        with pytest.raises(ss.SSError):
            bad()


def test_epilogue_oracle_by_hand():
    from oracle.fused_epilogue import activate, epilogue, epilogue_f32
    z = np.array([[-2.0, 0.5, 1.0, 3.0]])
    assert np.allclose(epilogue(z, bias=[1, 0, 0, 1], act="relu", residual=[[1, 1, 1, 1]]), [[1, 1.5, 2, 5]])
    assert np.allclose(epilogue(z, gated=True), [[-1.0, 3.0]]) and np.allclose(epilogue(z, act="relu", gated=True), [[0, 3]])
    assert np.allclose(activate(1.0, "silu"), 1 / (1 + math.exp(-1))) and np.allclose(activate(1.0, "gelu"), 0.8413447461)
    assert np.allclose(activate(1.0, "gelu_tanh"), 0.8411919906) and activate(-800.0, "silu") == 0
    assert np.array_equal(epilogue_f32(z, relu=True), np.maximum(z, 0).astype(np.float32))


@built
def test_epilogue_refusals():
    import structured_sparse_quantized_amd as ss
    odd = ctypes.c_void_p((1 << 20) + 8)

    def call(N=32, act=0, gated=0, res=None, ldr=32, y=ss.SS_BF16, ldy=32, sx=FAKE, bias=None, ws=None, n=0, M=8, Kc=256):
        return ss.lib.ss_spgemm_tiled_epilogue(0, M, N, Kc, ss.SS_I8, FAKE, FAKE, FAKE, Kc, sx, FAKE, bias, act, gated, res, ldr,
                                               y, FAKE, ldy, ws, n, None)

    assert call(y=ss.SS_I32) == ss.SS_ERR_DTYPE and call(act=5) == call(act=-1) == ss.SS_ERR_UNSUPPORTED
    assert call(N=31, gated=1) == call(ldy=31) == call(res=FAKE, ldr=31) == call(Kc=100) == call(n=-1) == ss.SS_ERR_SHAPE
    assert call(res=FAKE, ldr=40) == ss.SS_ERR_SHAPE  # Y itself with another stride
    assert call(res=odd) == call(bias=ctypes.c_void_p(2)) == ss.SS_ERR_ALIGN and call(sx=None) == ss.SS_ERR_NULL
    need = ss.spgemm_tiled_workspace_bytes(0, 40, 32, 256, "i8")
    assert need > 0 and call(M=40) == ss.SS_ERR_NULL and call(M=40, ws=FAKE, n=need - 1) == ss.SS_ERR_SHAPE
    assert call(M=0) == call(N=0) == ss.SS_OK
