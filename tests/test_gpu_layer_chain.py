"""A transformer layer run through the library without leaving it: quantise, query/key/value product with bias,
rotary positions in place, attention of packed sequences, output product onto the residual stream, gate product,
down product onto the residual stream; then the next tokens of the same sequences over their caches.

Each step is checked against its definition in float64 on the inputs that the step before really left, with the
tolerances of the operators' own tests: products 4e-5 of the sum of magnitudes, attention 2^-8 of its norm, and one
rounding of 2^-8 of the value each."""
import math

import numpy as np
import pytest
import torch

import oracle
from helpers import have_gpu, host
from oracle.attention import attention
from oracle.fused_epilogue import activate
from oracle.rotary import frequencies, rotary

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


def f64(t):
    return t.double().cpu().numpy() if t.dtype != torch.float8_e4m3fn else t.float().double().cpu().numpy()


class Linear:
    def __init__(self, ss, q, N, K, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        W = torch.randn((N, K), generator=g, device="cuda") / math.sqrt(K / 2)
        self.ss, self.q, self.N, self.K, self.Kc = ss, q, N, K, ss.lifted_k(K, 2)
        self.tv, self.tm, self.sw = ss.slide_decompose_tiled(W, 2, q)
        v, m, s = ss.slide_decompose(W, 2, q)
        self.W = oracle.decompress24(f64(v)[:, : self.Kc // 2], host(m), self.Kc)[:, :K]
        if s is not None:
            self.W = self.W * f64(s)[:, None]

    def __call__(self, x, **kw):
        M = x.shape[0]
        codes, sx = (x, None) if self.q == "bf16" else self.ss.quant_lift_act(x, 2, self.q)
        y = self.ss.spgemm_tiled_epilogue(self.ss.SS_SPARSE_W, M, self.N, self.Kc, self.tv, self.tm, codes, sx, self.sw, **kw)
        a = f64(codes)[:, : self.K] * (1.0 if sx is None else f64(sx)[:, None])
        self.z, self.mag = a @ self.W.T, np.abs(a) @ np.abs(self.W.T)
        return y


def near(got, exp, slack):
    tol = slack + 2.0 ** -8 * (np.abs(exp) + slack)
    assert (np.abs(f64(got) - exp) <= tol).all(), float((np.abs(f64(got) - exp) / tol).max())


@pytest.mark.parametrize("q", ["fp8", "i8", "bf16"])
def test_layer_then_next_tokens(ss, q):
    hidden, Hq, Hkv, D, ffn, cap = 512, 6, 2, 64, 768, 96
    lens = [33, 1, 70]
    B, T = len(lens), sum(lens)
    cum = np.concatenate([[0], np.cumsum(lens)]).tolist()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    H = Hq + Hkv
    qkv = Linear(ss, q, (H + Hkv) * D, hidden, 1)
    down_in = ffn
    o_w, gate, down = Linear(ss, q, hidden, 512, 2), Linear(ss, q, 2 * ffn, hidden, 3), Linear(ss, q, hidden, down_in, 4)
    bias = torch.randn((H + Hkv) * D, device="cuda")
    plan = dict(base=500000.0, scaling="smooth", factor=8.0, original=64, low=1.0, high=4.0)
    steps, ms = ss.rotary_steps(D, **plan)
    freq, _ = frequencies(D, **plan)
    kc, vc = (torch.full((B, cap, Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))

    def layer(x, pos, at):
        """x [T, hidden], the rows' positions and cache rows; returns the stream after the layer."""
        T = x.shape[0]
        row = qkv(x, bias=bias)
        near(row, qkv.z + f64(bias), 4e-5 * qkv.mag + 2.0 ** -22 * np.abs(qkv.z))
        heads = row.unflatten(1, (H + Hkv, D))
        turn = heads[:, :H]
        exp = rotary(f64(turn), pos.cpu().numpy(), freq, "half", ms)
        size = np.abs(f64(turn))
        size = size[..., : D // 2] + size[..., D // 2 :]
        ss.rotary(turn, pos, steps, mscale=ms, out=turn)
        near(turn, exp, 2.0 ** -21 * np.concatenate([size, size], -1))
        kc.flatten(0, 1)[at], vc.flatten(0, 1)[at] = heads[:, Hq:H], heads[:, H:]
        return heads

    def rest(x, mix):
        T = x.shape[0]
        wide = torch.zeros((T, 512), device="cuda", dtype=torch.bfloat16)  # heads side by side, padded to whole columns
        wide[:, : Hq * D] = mix.flatten(1)
        stream = x.clone()
        before = f64(stream)
        o_w(wide, residual=stream, out=stream)
        near(stream, o_w.z + before, 4e-5 * o_w.mag + 2.0 ** -22 * (np.abs(o_w.z) + np.abs(before)))
        mid = gate(stream, act="silu", gated=True)
        g, u = gate.z[:, 0::2], gate.z[:, 1::2]
        eg, eu = 4e-5 * gate.mag[:, 0::2], 4e-5 * gate.mag[:, 1::2]
        v = activate(g, "silu")
        near(mid, v * u, (1.13 * eg + 2.0 ** -18 * np.abs(v)) * (np.abs(u) + eu) + np.abs(v) * eu)
        before = f64(stream)
        down(mid, residual=stream, out=stream)
        near(stream, down.z + before, 4e-5 * down.mag + 2.0 ** -22 * (np.abs(down.z) + np.abs(before)))
        return stream

    def attend(heads, k, v, cq, ck, kl):
        mix = ss.attn(heads[:, :Hq], k, v, i32(cq), i32(ck), k_len=None if kl is None else i32(kl))
        exp = attention(f64(heads[:, :Hq]), np.nan_to_num(f64(k)), np.nan_to_num(f64(v)), cq, ck, kl)[0]
        assert np.linalg.norm(f64(mix) - exp) <= 2.0 ** -8 * np.linalg.norm(exp)
        return mix

    x = torch.randn((T, hidden), device="cuda").to(torch.bfloat16)
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens]).to(torch.int32)
    at = torch.cat([b * cap + torch.arange(n, device="cuda") for b, n in enumerate(lens)])
    heads = layer(x, pos, at)
    y = rest(x, attend(heads, heads[:, Hq:H], heads[:, H:], cum, cum, None))
    assert torch.isfinite(y.float()).all()
    starts = [b * cap for b in range(B + 1)]
    for step in range(2):  # one more token of each sequence
        x = torch.randn((B, hidden), device="cuda").to(torch.bfloat16)
        pos = i32([n + step for n in lens])
        at = torch.tensor([b * cap + n + step for b, n in enumerate(lens)], device="cuda")
        heads = layer(x, pos, at)
        mix = attend(heads, kc.flatten(0, 1), vc.flatten(0, 1), list(range(B + 1)), starts, [n + step + 1 for n in lens])
        assert torch.isfinite(rest(x, mix).float()).all()
