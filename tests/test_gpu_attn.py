"""ss_attn on the GPU against the float64 oracle: packed sequences, grouped heads, causal edges, empty rows and
sequences, caches with room, strided heads, partial heads of a tile, NaN where nothing is read, streams and graphs.

Tolerance. Products of bf16 values are exact in float32; the matrix core's sums keep 4e-5 of the sum of magnitudes
(as in the product tests), so a score is off by size * 4e-5 and a probability by twice that, relative (its own
power and the sum). Probabilities round to bf16 (2^-8), the second product again keeps 4e-5 of mass = sum p |v|,
exponents and powers in float32 add less than 2e-5 at scores of the sizes here; the output rounds by 2^-8 of itself.
The roundings of a row are independent, so over a whole tensor their root mean square (at most 2^-8 / sqrt(3)
each, two of them) stays below 2^-8 of its norm."""
import numpy as np
import pytest
import torch

from helpers import have_gpu
from oracle.attention import attention

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


def _cum(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(int).tolist()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _compare(o, lse, ref, norm=True):
    eo, el, mass, size = ref
    g = o.double().cpu().numpy()
    inside = ~np.isnan(eo)
    e = np.nan_to_num(size).T[:, :, None] * 8e-5 + 6e-5
    tol = np.nan_to_num(mass) * (2.0 ** -8 + e)
    tol = tol + 2.0 ** -8 * (np.abs(np.nan_to_num(eo)) + tol)
    err = np.abs(g - np.where(inside, eo, g))
    assert (err <= tol)[inside].all(), f"worst {np.nanmax(err / (tol + 1e-30)):.3g}"
    n = np.linalg.norm(np.nan_to_num(eo))
    if norm and n > 0:
        assert np.linalg.norm(np.where(inside, g - np.nan_to_num(eo), 0)) <= 2.0 ** -8 * n
    if lse is not None:
        gl = lse.double().cpu().numpy()
        lin = ~np.isnan(el)
        assert np.array_equal(np.isneginf(gl[lin]), np.isneginf(el[lin]))
        fin = np.isfinite(el)
        assert (np.abs(gl[fin] - el[fin]) <= (np.nan_to_num(size) * 4e-5 + 2e-5 + np.abs(np.where(fin, el, 0)) * 2.0 ** -22)[fin]).all()


def _run(ss, lq, lk, Hq, Hkv, D, causal, seed=0, scale=None, amp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Tq, Tk = sum(lq), sum(lk)
    q = (amp * torch.randn((Tq, Hq, D), generator=g, device="cuda")).to(torch.bfloat16)
    k, v = (torch.randn((Tk, Hkv, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cq, ck = _cum(lq), _cum(lk)
    lse = torch.full((Hq, Tq), 7.0, device="cuda")
    o = ss.attn(q, k, v, _i32(cq), _i32(ck), causal=causal, scale=scale, lse=lse)
    ref = attention(*(t.float().cpu().numpy() for t in (q, k, v)), cq, ck, None, causal, scale)
    _compare(o, lse, ref)
    return q, k, v, o, lse


LENS = [  # query and key lengths
    ([1], [1]), ([1], [65]), ([31], [31]), ([32], [32]), ([33], [33]), ([64], [64]), ([65], [65]), ([127], [200]),
    ([200], [127]), ([3], [0]), ([0, 5, 0, 1], [4, 0, 2, 1]), ([17, 1, 64, 0, 130], [17, 90, 64, 5, 131]), ([300], [300])]


@pytest.mark.parametrize("lq,lk", LENS, ids=lambda v: "-".join(map(str, v)))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 128), (7, 1, 64), (2, 2, 72)])
def test_packed(ss, lq, lk, causal, Hq, Hkv, D):
    _run(ss, lq, lk, Hq, Hkv, D, causal, seed=len(lq) + D)


@pytest.mark.parametrize("D", [8, 16, 40, 56, 64, 80, 96, 120, 128])
def test_head_sizes(ss, D):
    _run(ss, [70, 9], [70, 40], 3, 3, D, True, seed=D)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (28, 4), (32, 8), (71, 1), (12, 3)])
def test_grouped_heads(ss, Hq, Hkv):
    _run(ss, [40, 3], [40, 50], Hq, Hkv, 32, True, seed=Hq)


@pytest.mark.parametrize("Hq,Hkv,lq,lk", [(8, 1, [500, 37], [500, 90]), (2, 2, [400], [700]), (16, 2, [150, 1, 299], [150, 40, 310])])
def test_many_tiles(ss, Hq, Hkv, lq, lk):
    _run(ss, lq, lk, Hq, Hkv, 128, True, seed=3)


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (3, 1, 40), (2, 1, 128), (1, 1, 96)])
@pytest.mark.parametrize("lq,lk", [
    ([100], [1100]), ([1100], [1100]), ([1090], [1025]), ([70, 40], [2100, 63]), ([33, 200, 40], [3200, 0, 1]), ([40], [6000]),
    ([700], [1100]), ([1300, 1, 30], [2100, 1500, 0])])
@pytest.mark.parametrize("causal", [True, False])
def test_few_workgroups_split_the_keys(ss, lq, lk, causal, Hq, Hkv, D):
    q, k, v, o, lse = _run(ss, lq, lk, Hq, Hkv, D, causal, seed=D)
    again = torch.empty_like(lse)
    assert torch.equal(ss.attn(q, k, v, _i32(_cum(lq)), _i32(_cum(lk)), causal=causal, lse=again), o) and torch.equal(again, lse)


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D", [
    ([100], [6000], 8, 2, 128), ([16], [1030], 32, 8, 64), ([50, 1, 0, 77], [2100, 2500, 900, 4000], 4, 2, 72),
    ([130], [4100], 7, 1, 128), ([64, 64], [9000, 100], 4, 4, 40)])
def test_chunks_over_long_caches(ss, lq, lk, Hq, Hkv, D):
    for causal in (True, False):
        q, k, v, o, lse = _run(ss, lq, lk, Hq, Hkv, D, causal, seed=D)
        assert torch.equal(ss.attn(q, k, v, _i32(_cum(lq)), _i32(_cum(lk)), causal=causal), o)


def test_many_workgroups_of_long_keys(ss):
    _run(ss, [1300, 2000], [1300, 2000], 16, 16, 64, True, seed=8)
    _run(ss, [1500], [1500], 24, 24, 128, False, seed=9)


@pytest.mark.parametrize("D", [8, 64, 72, 128])
@pytest.mark.parametrize("lq,lk", [([1], [5000]), ([1, 1, 1], [3000, 1, 0]), ([4], [4097]), ([3, 1], [33, 6001]), ([2], [1])])
def test_few_rows_split_over_workgroups(ss, lq, lk, D):
    _run(ss, lq, lk, 7, 1, D, True, seed=D)
    _run(ss, lq, lk, 4, 4, D, False, seed=D + 1)


@pytest.mark.parametrize("amp", [1.0, 30.0, 800.0])
@pytest.mark.parametrize("lq,lk,D", [(200, 700, 128), (1500, 1500, 64), (90, 1300, 128), (5, 900, 64)])
def test_maxima_that_rise_along_the_keys(ss, lq, lk, D, amp):
    """Scores that grow (and for half of the rows fall) from key to key, by less and by far more than a float's range
    of exponents from one tile to the next."""
    g = torch.Generator(device="cuda").manual_seed(7)
    q = 0.1 * torch.randn((lq, 2, D), generator=g, device="cuda")
    k = 0.1 * torch.randn((lk, 2, D), generator=g, device="cuda")
    v = torch.randn((lk, 2, D), generator=g, device="cuda").to(torch.bfloat16)
    q[:, :, 0] = torch.where(torch.arange(lq, device="cuda") % 2 == 0, 1.0, -1.0)[:, None] * D ** 0.5
    k[:, :, 0] = torch.linspace(-amp, amp, lk, device="cuda")[:, None]
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    lse = torch.empty((2, lq), device="cuda")
    o = ss.attn(q, k, v, causal=True, lse=lse)
    _compare(o, lse, attention(*(t.float().cpu().numpy() for t in (q, k, v)), [0, lq], [0, lk], None, True, None), norm=False)


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D", [
    (200, 200, 2, 2, 128), (300, 333, 3, 1, 64), (150, 100, 2, 1, 40),  # tiles of many rows
    (100, 1100, 2, 1, 128), (1100, 1100, 1, 1, 64),  # the keys in two parts
    (6, 500, 4, 1, 128), (7, 90, 2, 2, 64), (4, 5000, 7, 1, 72)])  # few rows, one workgroup and several
def test_infinities_and_nan_reach_the_rows_that_see_them(ss, lq, lk, Hq, Hkv, D):
    g = torch.Generator(device="cuda").manual_seed(lq)
    q = torch.randn((lq, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((lk, Hkv, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    clean, lse, lse_k = ss.attn(q, k, v), torch.empty((Hq, lq), device="cuda"), torch.empty((Hq, lq), device="cuda")
    ss.attn(q, k, v, lse=lse)
    seen = (torch.arange(lq, device="cuda") + lk - lq + 1).clamp(0, lk)  # keys of a row
    for back in (1, 2, min(lq - 1, 5), min(lq - 1, 40)):
        j = max(lk - back, 0)
        rows = seen > j
        vb = v.clone()
        vb[j, :, 1], vb[j, :, 3], vb[j, :, D - 1] = float("nan"), float("inf"), -float("inf")
        o = ss.attn(q, k, vb, lse=lse_k)
        assert torch.equal(o[~rows], clean[~rows]) and torch.equal(lse_k, lse)
        other = [c for c in range(D) if c not in (1, 3, D - 1)]
        assert torch.equal(o[:, :, other], clean[:, :, other])
        assert o[rows][:, :, 1].isnan().all() and (o[rows][:, :, 3] == float("inf")).all()
        assert (o[rows][:, :, D - 1] == -float("inf")).all()
        kb = k.clone()
        kb[j, :, 2] = float("nan")
        o = ss.attn(q, kb, v, lse=lse_k)
        assert torch.equal(o[~rows], clean[~rows]) and torch.equal(lse_k[:, ~rows], lse[:, ~rows])
        assert o[rows].isnan().all() and lse_k[:, rows].isnan().all()


def test_own_workspace(ss):
    """A workspace of the stated size serves; its contents before do not matter."""
    q = torch.randn((2, 8, 64), device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((9000, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    need = ss.attn_workspace_bytes(2, 9000, 1, 8, 2, 64)
    assert need > 0
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    o = ss.attn(q, k, v, workspace=ws[:need])
    assert torch.equal(o, ss.attn(q, k, v)) and (ws[need:] == 255).all()
    with pytest.raises(ss.SSError):
        ss.attn(q, k, v, workspace=ws[: need - 1])


def test_offsets_beyond_32_bits(ss):
    """Sequences behind more than 2^31 elements of keys, and one sequence longer than that."""
    far = 2200000
    k, v = (torch.zeros((far, 8, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(3)
    k[-900:], v[-900:] = (torch.randn((900, 8, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    for lq in (1, 200):
        q = torch.randn((lq, 16, 128), generator=g, device="cuda").to(torch.bfloat16)
        o = ss.attn(q, k, v, _i32([0, lq]), _i32([far - 900, far]))
        ref = attention(q.float().cpu().numpy(), *(t[-900:].float().cpu().numpy() for t in (k, v)), [0, lq], [0, 900])
        _compare(o, None, ref)
    del k, v
    n = 17000000
    k, v = (torch.zeros((n, 1, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn((1, 2, 128), generator=g, device="cuda").to(torch.bfloat16)
    k[-100:, 0] = 6 * q.float().mean(1).to(torch.bfloat16)
    v[-100:] = torch.randn((100, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    o = ss.attn(q, k, v)
    s = k[-100:, 0].double() @ q[0].double().T * 128 ** -0.5  # the other keys score 0
    e = torch.exp(s)
    p = e / (e.sum(0) + (n - 100))
    want = (p.T[:, :, None] * v[None, -100:, 0].double()).sum(1)
    mass = (p.T[:, :, None] * v[None, -100:, 0].double().abs()).sum(1)
    assert float(p.sum(0).min()) > 0.5  # the last keys carry the row
    assert ((o[0].double() - want).abs() <= mass * (2.0 ** -8 + float(s.abs().max()) * 8e-5 + 6e-5) + 2.0 ** -8 * want.abs()).all()


def test_large_scores(ss):
    """Scores far apart: the running maximum rises many times and most powers vanish."""
    _run(ss, [130], [260], 2, 1, 64, True, seed=5, amp=8.0)
    _run(ss, [130], [260], 2, 1, 64, False, seed=6, scale=1e-4)


def test_rising_maximum(ss):
    """Keys ordered so that every tile raises the maximum: the earlier sums are rescaled each time."""
    D, n = 64, 640
    q = torch.ones((4, 2, D), device="cuda").to(torch.bfloat16)
    k = torch.linspace(-8, 8, n, device="cuda")[:, None, None].expand(n, 1, D).to(torch.bfloat16)
    v = torch.randn((n, 1, D), device="cuda").to(torch.bfloat16)
    for kk in (k, k.flip(0)):
        kk = kk.contiguous()
        o = ss.attn(q, kk, v, causal=False)
        _compare(o, None, attention(*(t.float().cpu().numpy() for t in (q, kk, v)), [0, 4], [0, n], None, False))


def test_caches_with_room(ss):
    """Single tokens and short chunks over caches: k_len keys in use, NaN in the room behind them."""
    B, cap, Hq, Hkv, D = 5, 300, 8, 2, 128
    used = [1, 300, 77, 0, 129]
    k, v = (torch.randn((B, cap, Hkv, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    for b, n in enumerate(used):
        k[b, n:], v[b, n:] = float("nan"), float("nan")
    kf, vf = k.flatten(0, 1), v.flatten(0, 1)
    ck = [b * cap for b in range(B + 1)]
    for lq in ([1] * B, [3, 1, 4, 2, 1], [40] * B):
        q = torch.randn((sum(lq), Hq, D), device="cuda").to(torch.bfloat16)
        lse = torch.empty((Hq, sum(lq)), device="cuda")
        o = ss.attn(q, kf, vf, _i32(_cum(lq)), _i32(ck), k_len=_i32(used), lse=lse)
        ref = attention(q.float().cpu().numpy(), np.nan_to_num(kf.float().cpu().numpy()), np.nan_to_num(vf.float().cpu().numpy()),
                        _cum(lq), ck, used)
        _compare(o, lse, ref)


def test_strided_heads_and_untouched_rows(ss):
    """Heads inside a projection's output, head-major caches, an output inside another tensor; query rows before
    the first and behind the last sequence, and NaN keys between sequences."""
    T, Hq, Hkv, D = 90, 6, 2, 64
    row = torch.randn((T, (Hq + 2 * Hkv) * D), device="cuda").to(torch.bfloat16).unflatten(1, (Hq + 2 * Hkv, D))
    q = row[:, :Hq]
    kc = torch.full((Hkv, 120, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    vc = kc.clone()
    cq, ck, kl = [4, 34, 80], [10, 60, 120], [41, 50]
    kc[:, 10:51], vc[:, 10:51] = torch.randn((2, Hkv, 41, D), device="cuda").to(torch.bfloat16)
    kc[:, 60:110], vc[:, 60:110] = torch.randn((2, Hkv, 50, D), device="cuda").to(torch.bfloat16)
    dst = torch.full((T, Hq + 1, D + 8), 3.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((Hq, T), 3.0, device="cuda")
    out = dst[:, 1:, :D]
    k, v = kc.transpose(0, 1), vc.transpose(0, 1)
    assert ss.attn(q, k, v, _i32(cq), _i32(ck), k_len=_i32(kl), out=out, lse=lse) is out
    ref = attention(q.float().cpu().numpy(), *(np.nan_to_num(t.float().cpu().numpy()) for t in (k, v)), cq, ck, kl)
    _compare(out, lse, ref)
    assert (dst[:, 0] == 3).all() and (dst[:, :, D:] == 3).all() and (dst[:4] == 3).all() and (dst[80:] == 3).all()
    assert (lse[:, :4] == 3).all() and (lse[:, 80:] == 3).all()


def test_shared_keys_by_stride_zero(ss):
    """k and v expanded over heads and over tokens (stride 0)."""
    q = torch.randn((20, 4, 32), device="cuda").to(torch.bfloat16)
    k = torch.randn((50, 1, 32), device="cuda").to(torch.bfloat16).expand(50, 4, 32)
    v = torch.randn((1, 4, 32), device="cuda").to(torch.bfloat16).expand(50, 4, 32)
    o = ss.attn(q, k, v)
    _compare(o, None, attention(*(t.float().cpu().numpy() for t in (q, k, v)), [0, 20], [0, 50]), norm=False)


def test_bad_bounds_stay_inside(ss):
    """Bounds past the tensors are clamped to them; nothing outside is read or written."""
    q, k, v = (torch.randn((40, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(3))
    o = ss.attn(q, k, v, _i32([0, 4000]), _i32([-5, 1 << 30]), k_len=_i32([1 << 30]))
    assert torch.equal(o, ss.attn(q, k, v))
    ss.attn(q, k, v, _i32([30, 10, 50]), _i32([20, 5, 90]))
    torch.cuda.synchronize()


def test_many_sequences(ss):
    rng = np.random.default_rng(1)
    lq, lk = rng.integers(0, 4, 300).tolist(), rng.integers(0, 9, 300).tolist()
    _run(ss, lq, lk, 2, 1, 16, True, seed=9)
    _run(ss, [1] * 70, [3] * 70, 2, 1, 16, False, seed=10)


def test_repeatable_on_another_stream_and_in_a_graph(ss):
    """The same bits from call to call, on another stream, and from a graph replayed with other inputs, lengths
    and eager work between."""
    for lq, cap in (([1] * 6, 900), ([50] * 3, 120)):
        B = len(lq)
        q = torch.randn((sum(lq), 8, 128), device="cuda").to(torch.bfloat16)
        k, v = (torch.randn((B * cap, 2, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
        cq, ck, kl = _i32(_cum(lq)), _i32([b * cap for b in range(B + 1)]), _i32([cap - 7 * b for b in range(B)])
        first = ss.attn(q, k, v, cq, ck, k_len=kl)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = ss.attn(q, k, v, cq, ck, k_len=kl)
        s.synchronize()
        assert torch.equal(first, other)
        graphs, outs = [], []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(ss.attn(q, k, v, cq, ck, k_len=kl))
            graphs.append(graph)
        for rep in range(3):
            q.copy_(torch.randn_like(q))
            kl.fill_(cap - 100 * rep // 2 - 1)
            for graph in graphs:
                graph.replay()
            want = ss.attn(q, k, v, cq, ck, k_len=kl)
            torch.cuda.synchronize()
            assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_empty(ss):
    z = torch.empty((0, 4, 64), device="cuda", dtype=torch.bfloat16)
    q = torch.randn((5, 4, 64), device="cuda").to(torch.bfloat16)
    assert ss.attn(z, q, q).shape == (0, 4, 64)
    lse = torch.empty((4, 5), device="cuda")
    assert (ss.attn(q, z, z, lse=lse) == 0).all() and torch.isneginf(lse).all()
    assert (ss.attn(q, z, z, _i32([0, 2, 5]), _i32([0, 0, 0])) == 0).all()


def test_refused(ss):
    q = torch.zeros((5, 4, 64), device="cuda", dtype=torch.bfloat16)
    for bad in (lambda: ss.attn(q, q[:, :3], q[:, :3]), lambda: ss.attn(q, q, q, _i32([0, 5]).long()),
                lambda: ss.attn(q, q, q, _i32([0, 5]), _i32([0, 2, 5])), lambda: ss.attn(q, q, q, k_len=_i32([1, 2])),
                lambda: ss.attn(q[..., :60], q[..., :60], q[..., :60]), lambda: ss.attn(q, q, q[:4]),
                lambda: ss.attn(q, q, q, scale=0.0), lambda: ss.attn(q, q, q, out=q.float()),
                lambda: ss.attn(q, q, q, _i32([])), lambda: ss.attn(q, q, q, _i32([0, 2, 5]))):
        with pytest.raises(ss.SSError):
            bad()
