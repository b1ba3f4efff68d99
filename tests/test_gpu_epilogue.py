"""ss_spgemm_tiled_epilogue on the GPU against the oracle: every kernel the product takes (row-block, split-K,
256 x 128 tiles, wide 256 x 128 and 256 x 256 of eight and four waves), both sides, every operand and output type,
bias, each activation, gate, residual (also in place), ragged sizes, padded leading dimensions, streams and graphs.

Tolerance. z carries the product's own error (INT8: none; else 4e-5 of the sum of magnitudes, as in the product
tests) and three roundings of at most 2^-24 of |scaled| + |bias|: ez. No activation is steeper than 1.13. The
exponential forms add |v| (2^-19 + |u| 2^-22) where the chip's exponential is taken (its own error and that of
its argument's rounding, u the exponent), erf 2^-22 |z|; a gate multiplies two such values; the sum with the
residual rounds by 2^-24 of it, the output by 2^-8 (bf16) or 2^-24 (f32) of itself."""
import math

import numpy as np
import pytest
import torch

import oracle
from helpers import bf16_to_f64, have_gpu, host
from oracle.fused_epilogue import activate, epilogue, epilogue_f32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


class Problem:
    """Operands of one product, and in float64 the scaled sums and sums of magnitudes of some token rows."""

    def __init__(self, ss, side, q, M, N, K, seed=0, rows=48):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.M, self.N, self.q, self.side = M, N, q, ss.SS_SPARSE_W if side == "W" else ss.SS_SPARSE_X
        self.Kc = Kc = ss.lifted_k(K, 2)  # also the row stride, so that rows start on 16 bytes at any K
        W = (torch.randn((N, Kc), generator=g, device="cuda") / math.sqrt(K / 2))[:, :K]
        X = torch.randn((M, Kc), generator=g, device="cuda").to(torch.bfloat16)[:, :K]
        if side == "W":
            v, m, self.sw = ss.slide_decompose(W, 2, q)
            if q == "bf16":
                d, self.sx = torch.zeros((M, Kc), dtype=torch.bfloat16, device="cuda"), None
                d[:, :K] = X
            else:
                d, self.sx = ss.quant_lift_act(X, 2, q)
        else:
            v, m, self.sx = ss.prune24_act(X, q)
            if q == "bf16":
                d, self.sw = torch.zeros((N, Kc), dtype=torch.bfloat16, device="cuda"), None
                d[:, :K] = W.to(torch.bfloat16)
            else:
                d, self.sw = ss.quant_lift_act(W, 2, q)
        self.tv, self.tm = ss.pack_sparse(v, m)
        self.dense = d
        self.rows = np.unique(np.concatenate([np.arange(min(M, 3)), np.linspace(0, M - 1, rows).astype(int)]))
        dec = {"i8": lambda t: t.double(), "fp8": lambda t: t.float().double(), "bf16": lambda t: t.double()}[q]
        sp = torch.from_numpy(oracle.decompress24(dec(v).cpu().numpy()[:, : Kc // 2], host(m), Kc))
        dn = dec(d).cpu()
        a, b = (dn[self.rows], sp) if side == "W" else (sp[self.rows], dn)
        acc, mag = (a @ b.T).numpy(), (a.abs() @ b.abs().T).numpy()
        sx = 1.0 if self.sx is None else self.sx.double().cpu().numpy()[self.rows, None]
        sw = 1.0 if self.sw is None else self.sw.double().cpu().numpy()[None, :]
        self.scaled, self.mag = acc * sx * sw, mag * np.abs(sx * sw)
        if q == "i8":  # step by step in float32
            f = acc.astype(np.float32) * np.asarray(sx, np.float32)
            self.f32 = f * np.asarray(sw, np.float32)

    def run(self, ss, **kw):
        return ss.spgemm_tiled_epilogue(self.side, self.M, self.N, self.Kc, self.tv, self.tm, self.dense, self.sx, self.sw, **kw)

    def check(self, ss, bias=None, act="none", gated=False, residual=None, y="bf16", **kw):
        Y = self.run(ss, bias=bias, act=act, gated=gated, residual=residual, y_dtype=y, **kw)
        assert Y.shape == (self.M, self.N // 2 if gated else self.N)
        got = Y[self.rows].double().cpu().numpy()
        b = None if bias is None else bias.double().cpu().numpy()
        r = None if residual is None else residual[self.rows].double().cpu().numpy()
        if self.q == "i8" and act in ("none", "relu"):  # exact
            e = epilogue_f32(self.f32, b, act == "relu", gated, r)
            if y == "bf16":
                e = bf16_to_f64(oracle.f32_to_bf16_bits_rne(e))
            assert np.array_equal(got, np.asarray(e, np.float64))
            return Y
        exp = epilogue(self.scaled, b, act, gated, r)
        z = self.scaled + (0 if b is None else b)
        ez = 3 * 2.0 ** -24 * (np.abs(self.scaled) + (0 if b is None else np.abs(b))) + (0 if self.q == "i8" else 4e-5) * self.mag
        v = activate(z, act)
        u = np.abs(z) if act == "silu" else 1.6 * np.abs(z + 0.044715 * z ** 3)
        ev = 1.13 * ez + {"none": 0, "relu": 0, "gelu": 2.0 ** -22 * np.abs(z)}.get(act, np.abs(v) * (2.0 ** -19 + u * 2.0 ** -22))
        if gated:
            ev = ev[:, 0::2] * np.abs(z[:, 1::2]) + np.abs(v[:, 0::2]) * ez[:, 1::2] + 2.0 ** -24 * np.abs(v[:, 0::2] * z[:, 1::2])
        tol = ev + 2.0 ** -24 * np.abs(exp)
        tol = tol + (2.0 ** -8 if y == "bf16" else 2.0 ** -24) * (np.abs(exp) + tol) + 1e-30
        assert (np.abs(got - exp) <= tol).all(), float((np.abs(got - exp) / tol).max())
        return Y


def _extras(p, gated, y, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if y == "bf16" else torch.float32
    return (torch.randn(p.N, generator=g, device="cuda"),
            torch.randn((p.M, p.N // 2 if gated else p.N), generator=g, device="cuda").to(dt))


SMALL = [(1, 16, 256), (1, 4608, 512), (3, 50, 300), (16, 130, 700), (17, 514, 512), (48, 1000, 1100), (64, 128, 256), (65, 600, 300),
         (200, 130, 600)]


@pytest.mark.parametrize("M,N,K", SMALL)
@pytest.mark.parametrize("side", ["W", "X"])
@pytest.mark.parametrize("q", ["i8", "fp8", "bf16"])
def test_small(ss, M, N, K, side, q):
    p = Problem(ss, side, q, M, N, K, seed=M + N)
    for i, act in enumerate(ACTS):
        y = "bf16" if (i + M) % 2 else "f32"
        for gated in (False, True):
            b, r = _extras(p, gated, y)
            p.check(ss, bias=b, act=act, gated=gated, residual=r, y=y)
        b, r = _extras(p, False, y)
        p.check(ss, act=act, y=y)
        p.check(ss, act=act, bias=b, y=y)
        p.check(ss, act=act, residual=r, y=y)


@pytest.mark.parametrize("side,q,M,N,K", [
    ("W", "i8", 2200, 4097, 256), ("W", "fp8", 2200, 4098, 500), ("W", "bf16", 2200, 4096, 256),  # wide 256 x 128
    ("X", "i8", 4100, 2305, 256), ("X", "fp8", 4100, 2306, 500), ("X", "bf16", 4096, 2304, 256),
    ("W", "i8", 4090, 8191, 256), ("W", "fp8", 4096, 8192, 512), ("W", "bf16", 4090, 8190, 256),  # wide 256 x 256, eight waves
    ("W", "i8", 2560, 4096, 8448), ("W", "fp8", 2559, 4094, 8448), ("W", "bf16", 2560, 4096, 4352),  # four waves
    ("W", "i8", 300, 2000, 600), ("X", "fp8", 300, 2000, 600)])  # 256 x 128 tiles, one per CU
def test_prefill(ss, side, q, M, N, K):
    p = Problem(ss, side, q, M, N, K, seed=N)
    for act, gated, y in (("none", False, "bf16"), ("silu", True, "bf16"), ("gelu", False, "f32"), ("relu", True, "f32"),
                          ("gelu_tanh", False, "bf16")):
        if gated and N % 2:
            continue
        b, r = _extras(p, gated, y)
        Y = p.check(ss, bias=b, act=act, gated=gated, residual=r, y=y)
        assert torch.equal(Y, p.run(ss, bias=b, act=act, gated=gated, residual=r, y_dtype=y))
    p.check(ss, act="silu")


@pytest.mark.parametrize("side,q,M,N,K", [
    ("W", "i8", 65, 4098, 600), ("W", "fp8", 130, 2047, 256), ("W", "bf16", 200, 1000, 1000),  # widths of 32
    ("W", "i8", 350, 2050, 256), ("W", "fp8", 250, 4094, 512), ("W", "bf16", 800, 1100, 128),  # 64
    ("W", "i8", 400, 4097, 256), ("W", "fp8", 385, 3970, 640), ("W", "bf16", 1000, 2044, 256),  # 128
    ("X", "i8", 500, 1001, 600), ("X", "fp8", 1500, 333, 256), ("X", "bf16", 777, 900, 500),
    ("X", "i8", 1030, 990, 256), ("X", "fp8", 1100, 1601, 256), ("X", "bf16", 2047, 250, 256),
    ("W", "fp8", 2999, 1030, 256), ("X", "i8", 1100, 2600, 500),  # three of width 64 a CU
    ("W", "i8", 10, 16390, 256), ("W", "fp8", 16, 12290, 256), ("W", "bf16", 64, 16450, 128), ("W", "fp8", 30, 20001, 512)])
def test_small_tiles(ss, side, q, M, N, K):
    p = Problem(ss, side, q, M, N, K, seed=N)
    for act, gated, y in (("none", False, "bf16"), ("silu", True, "bf16"), ("gelu", False, "f32"), ("relu", True, "f32")):
        if gated and N % 2:
            continue
        b, r = _extras(p, gated, y)
        Y = p.check(ss, bias=b, act=act, gated=gated, residual=r, y=y)
        assert torch.equal(Y, p.run(ss, bias=b, act=act, gated=gated, residual=r, y_dtype=y))
    p.check(ss, act="silu")
    if M > 64:
        plain = ss.spgemm_tiled(p.side, M, N, p.Kc, p.tv, p.tm, p.dense, p.sx, p.sw, "f32")
        assert torch.equal(plain, p.run(ss, y_dtype="f32"))


@pytest.mark.parametrize("M,N,K", [(5, 300, 256), (40, 600, 512), (300, 300, 256), (2200, 4096, 256)])
def test_equals_the_plain_product_without_extras(ss, M, N, K):
    for q in ("i8", "fp8"):
        p = Problem(ss, "W", q, M, N, K, seed=2)
        for y in ("bf16", "f32"):
            plain = ss.spgemm_tiled(p.side, M, N, p.Kc, p.tv, p.tm, p.dense, p.sx, p.sw, y)
            assert torch.equal(plain, p.run(ss, y_dtype=y))


@pytest.mark.parametrize("M,N", [(3, 70), (40, 600), (300, 130), (2200, 4096)])
@pytest.mark.parametrize("gated", [False, True])
def test_strides_and_residual_in_place(ss, M, N, gated):
    p = Problem(ss, "W", "fp8", M, N, 256, seed=3)
    cols = N // 2 if gated else N
    for pad in (8, 3):  # rows on and off 16-byte places
        for y, dt in (("bf16", torch.bfloat16), ("f32", torch.float32)):
            buf = torch.full((M, cols + pad), 9.0, device="cuda", dtype=dt)
            res = torch.randn((M, cols + pad + 8), device="cuda").to(dt)[:, :cols]
            out = buf[:, :cols]
            assert p.check(ss, act="silu", gated=gated, residual=res, y=y, out=out) is out and (buf[:, cols:] == 9).all()
            stream = torch.empty_like(buf)  # the residual stream updated in place
            stream[:, :cols] = res
            p.run(ss, act="silu", gated=gated, residual=stream[:, :cols], y_dtype=y, out=stream[:, :cols])
            assert torch.equal(stream[:, :cols], out)


def test_large_arguments(ss):
    """Gates and activations far out: no overflow, zeros and identities where they belong."""
    p = Problem(ss, "W", "i8", 70, 512, 256, seed=4)
    z = torch.linspace(-300, 300, 512, device="cuda")
    for act in ACTS:
        for y in ("bf16", "f32"):
            p.check(ss, bias=z, act=act, y=y)
            assert torch.isfinite(p.run(ss, bias=100 * z, act=act, y_dtype=y)).all()


@pytest.mark.parametrize("side,M,N", [("W", 3, 70), ("W", 40, 600), ("W", 300, 602), ("X", 100, 90), ("W", 2200, 4096)])
def test_nan_stays_in_its_column(ss, side, M, N):
    p = Problem(ss, side, "fp8", M, N, 256, seed=6)
    b = torch.randn(N, device="cuda")
    nan = b.clone()
    nan[[6, N - 3]] = float("nan")  # a gate (even) and a value (odd)
    for act in ACTS:
        for gated in (False, True):
            for y in ("bf16", "f32"):
                kw = dict(act=act, gated=gated, y_dtype=y)
                got, clean = p.run(ss, bias=nan, **kw), p.run(ss, bias=b, **kw)
                bad = torch.zeros(got.shape[1], dtype=torch.bool, device="cuda")
                bad[[6 >> gated, (N - 3) >> gated]] = True
                assert got[:, bad].isnan().all() and torch.equal(got[:, ~bad], clean[:, ~bad])


def test_workspace_stream_and_graph(ss):
    for M, N in ((40, 600), (2200, 4096)):
        p = Problem(ss, "W", "fp8", M, N, 512, seed=5)
        b, r = _extras(p, False, "bf16")
        kw = dict(bias=b, act="gelu", residual=r)
        want = p.run(ss, **kw)
        need = ss.spgemm_tiled_workspace_bytes(p.side, M, N, p.Kc, "fp8")
        assert (need > 0) == (M == 40)
        if need:
            ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")
            assert torch.equal(p.run(ss, workspace=ws[:need], **kw), want) and (ws[need:] == 255).all()
            with pytest.raises(ss.SSError):
                p.run(ss, workspace=ws[: need - 16], **kw)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = p.run(ss, **kw)
        s.synchronize()
        assert torch.equal(other, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = p.run(ss, **kw)
        for _ in range(3):
            r.copy_(torch.randn_like(r))
            b.add_(1)
            graph.replay()
            eager = p.run(ss, **kw)
            torch.cuda.synchronize()
            assert torch.equal(out, eager)


@pytest.mark.parametrize("gated,N", [(False, 28672), (False, 28671), (True, 57344)])
def test_outputs_beyond_32_bits(ss, gated, N):
    M, K, cols = 80000, 256, N // 2 if gated else N
    p = Problem(ss, "W", "fp8", 400, N, K, seed=8)
    dense, sx = p.dense.repeat(M // 400, 1), p.sx.repeat(M // 400)
    res = torch.zeros((M, cols), device="cuda", dtype=torch.bfloat16)
    res[-400:] = torch.randn((400, cols), device="cuda").to(torch.bfloat16)
    want = p.run(ss, act="relu", gated=gated, residual=res[-400:].clone())
    y = ss.spgemm_tiled_epilogue(p.side, M, N, p.Kc, p.tv, p.tm, dense, sx, p.sw, act="relu", gated=gated, residual=res)
    assert torch.equal(y[-400:], want)


def test_refused(ss):
    p = Problem(ss, "W", "i8", 8, 32, 256)
    one = torch.zeros((8, 32), device="cuda")
    for kw in (dict(act="swish"), dict(y_dtype="i32"), dict(bias=torch.zeros(31, device="cuda")), dict(bias=one[0].bfloat16()),
               dict(residual=one), dict(residual=one[:, :31].bfloat16()), dict(gated=True, out=one[:4].bfloat16()),
               dict(out=one), dict(bias=torch.zeros(32))):
        with pytest.raises(ss.SSError):
            p.run(ss, **kw)
    odd = Problem(ss, "W", "i8", 8, 33, 256)
    with pytest.raises(ss.SSError):
        odd.run(ss, gated=True)
    buf = torch.zeros((8, 40), device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ss.SSError):  # the residual in place through another stride
        p.run(ss, residual=buf[:, :32], out=buf.flatten()[:256].view(8, 32))
    empty = ss.spgemm_tiled_epilogue(p.side, 0, 32, p.Kc, p.tv, p.tm, p.dense[:0], p.sx[:0], p.sw)
    assert empty.shape == (0, 32)
