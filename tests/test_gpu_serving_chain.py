"""A transformer layer as a server runs it, without leaving the library: norm and quantisation, query/key/value product, turn and
write into the paged cache, attention over the pages, output product, norm of the sum with the residual, gated product, down
product, whose output the next layer's norm adds. A packed prompt of several sequences (with and without a window), then
single tokens, then a few drafted tokens at once; pages behind the window are given back.

Each step is checked against its definition in float64 on the inputs that the step before really left, with the tolerances of
the operators' own tests: the norm's outputs bit for bit, products 4e-5 of the sum of magnitudes and one rounding, the turn
2^-21 of the pair's magnitudes and one rounding, attention 2^-8 of its norm."""
import math

import numpy as np
import pytest
import torch

import oracle
from helpers import have_gpu, host
from oracle.norm import codes, rmsnorm
from oracle.fused_epilogue import activate
from oracle.rotary import frequencies, rotary
from oracle.windowed import packed, paged

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


def f64(t):
    return (t.float() if t.dtype == torch.float8_e4m3fn else t).double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Linear:
    """Sparse weights of pattern (2n-2):2n and the product with activations that the norm has prepared."""

    def __init__(self, ss, q, n, N, K, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        W = torch.randn((N, K), generator=g, device="cuda") / math.sqrt(K)
        self.ss, self.N, self.Kc = ss, N, ss.lifted_k(K, n)
        self.tv, self.tm, self.sw = ss.slide_decompose_tiled(W, n, q)
        v, m, s = ss.slide_decompose(W, n, q)
        self.W = oracle.decompress24(f64(v)[:, : self.Kc // 2], host(m), self.Kc) * f64(s)[:, None]  # over K'

    def __call__(self, x, sx, **kw):
        y = self.ss.spgemm_tiled_epilogue(self.ss.SS_SPARSE_W, x.shape[0], self.N, self.Kc, self.tv, self.tm, x, sx, self.sw, **kw)
        a = f64(x) * f64(sx)[:, None]
        self.z, self.mag = a @ self.W.T, np.abs(a) @ np.abs(self.W.T)
        return y


def near(got, exp, slack):
    tol = slack + 2.0 ** -8 * (np.abs(exp) + slack)
    assert (np.abs(f64(got) - exp) <= tol).all(), float((np.abs(f64(got) - exp) / tol).max())


@pytest.mark.parametrize("q,n", [("fp8", 2), ("i8", 4)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (40, 3)])
def test_prompt_tokens_and_drafts(ss, q, n, window, sinks):
    hidden, Hq, Hkv, D, ffn, page, cols = 512, 6, 2, 64, 768, 16, 12
    lens = [33, 1, 70]
    B = len(lens)
    H = Hq + 2 * Hkv
    qkv, o_w = Linear(ss, q, n, H * D, hidden, 1), Linear(ss, q, n, hidden, Hq * D, 2)
    gate, down = Linear(ss, q, n, 2 * ffn, hidden, 3), Linear(ss, q, n, hidden, ffn, 4)
    w1, w2 = ((0.5 + torch.rand(hidden, device="cuda")).to(torch.bfloat16) for _ in range(2))
    steps, ms = ss.rotary_steps(D, base=500000.0)
    freq, _ = frequencies(D, base=500000.0)
    pools = [torch.full((B * cols + 5, page, Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    rng = np.random.default_rng(0)
    table = rng.permutation(B * cols + 5)[: B * cols].reshape(B, cols)

    def prepare(x, w, residual):
        """The norm's three outputs, bit for bit."""
        before = x.float().cpu().numpy(), residual.float().cpu().numpy()
        y, sx, r = ss.rmsnorm_act(x, w, 1e-5, residual=residual, n=n, y_dtype=q, sum_out=residual)
        z, total = rmsnorm(before[0], w.float().cpu().numpy(), 1e-5, before[1])
        c, s = codes(z, n, q)
        assert np.array_equal(host(y), c) and np.array_equal(host(sx), s) and np.array_equal(r.float().cpu().numpy(), total)
        assert r.data_ptr() == residual.data_ptr()
        return y, sx

    def layer(x, stream, at, cu, prompt):
        """x and stream [T, hidden]; at: places of the tokens; returns what the next norm adds to the stream."""
        row = qkv(*prepare(x, w1, stream))
        near(row, qkv.z, 4e-5 * qkv.mag + 2.0 ** -22 * np.abs(qkv.z))
        heads = row.unflatten(1, (H, D))
        qh, kh, vh = heads[:, :Hq], heads[:, Hq : Hq + Hkv], heads[:, Hq + Hkv :]
        ek, eq = rotary(f64(kh), np.array(at), freq), rotary(f64(qh), np.array(at), freq)
        size = [np.abs(f64(t)) for t in (qh, kh)]
        size = [np.concatenate([s[..., : D // 2] + s[..., D // 2 :]] * 2, -1) for s in size]
        pages = i32(table.tolist())
        ss.paged_store(kh, vh, i32(at), *pools, pages, cu=i32(cu), q=qh, steps=steps, mscale=ms, q_out=qh)
        near(qh, eq, 2.0 ** -21 * size[0])
        seq = [b for b in range(B) for _ in range(cu[b + 1] - cu[b])]
        e = torch.tensor([table[b, p // page] for b, p in zip(seq, at)], device="cuda")
        p = torch.tensor([p % page for p in at], device="cuda")
        near(pools[0][e, p], ek, 2.0 ** -21 * size[1])
        assert torch.equal(pools[1][e, p], vh)
        n_keys = [at[cu[b + 1] - 1] + 1 for b in range(B)]
        w, s = window or 0, sinks
        if prompt:  # the turned keys as the cache holds them
            mix = ss.attn(qh, pools[0][e, p], vh, i32(cu), i32(cu), window=window, sinks=sinks)
            exp = packed(f64(qh), f64(pools[0][e, p]), f64(vh), cu, cu, None, True, w, s)[0]
            assert np.linalg.norm(f64(mix) - exp) <= 2.0 ** -8 * np.linalg.norm(exp)
        mix = ss.attn_paged(qh, *pools, pages, i32(n_keys), cu_q=i32(cu), window=window, sinks=sinks)
        exp = paged(f64(qh), *(f64(t) for t in pools), table.tolist(), n_keys, cu, True, w, s)[0]
        assert np.linalg.norm(f64(mix) - exp) <= 2.0 ** -8 * np.linalg.norm(exp)
        a, sa = ss.quant_lift_act(mix.flatten(1), n, q)
        out = o_w(a, sa)
        near(out, o_w.z, 4e-5 * o_w.mag + 2.0 ** -22 * np.abs(o_w.z))
        mid = gate(*prepare(out, w2, stream), act="silu", gated=True)
        g, u = gate.z[:, 0::2], gate.z[:, 1::2]
        eg, eu = 4e-5 * gate.mag[:, 0::2], 4e-5 * gate.mag[:, 1::2]
        v = activate(g, "silu")
        near(mid, v * u, (1.13 * eg + 2.0 ** -18 * np.abs(v)) * (np.abs(u) + eu) + np.abs(v) * eu)
        y = down(*ss.quant_lift_act(mid, n, q))
        near(y, down.z, 4e-5 * down.mag + 2.0 ** -22 * np.abs(down.z))
        return y

    def tokens(count):
        return [torch.randn((count, hidden), device="cuda").to(torch.bfloat16) for _ in range(2)]

    have = [0] * B
    for new in (lens, [1] * B, [1] * B, [4, 2, 7], [1] * B):
        x, stream = tokens(sum(new))
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        at = [have[b] + i for b in range(B) for i in range(new[b])]
        y = layer(x, stream, at, cu, have == [0] * B)
        assert torch.isfinite(y.float()).all()
        have = [a + b for a, b in zip(have, new)]
        if window:  # pages that no later token sees are given back, and what others write there meets no row
            for b in range(B):
                for i in range(-(-sinks // page), max(have[b] - window + 1, 0) // page):
                    if table[b, i] >= 0:
                        for t in pools:
                            t[table[b, i]] = float("nan")
                        table[b, i] = -1
