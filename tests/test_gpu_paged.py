"""ss_paged_store and ss_attn_paged on the GPU against the float64 oracles: pages of any size in any order, entries that name no
page, lengths from zero on, several tokens a sequence, windows with first tokens, runs that cut tiles and sequences anywhere,
NaN wherever nothing is to be read, caches beyond 32-bit offsets, streams, workspaces and graphs.

Tolerances of the attention are those of the packed attention's tests: scores keep 4e-5 of the sum of magnitudes, a
probability twice that, relative, plus its rounding to bf16 (2^-8); the output rounds by 2^-8 of itself; over a tensor the
roundings of a row are independent and stay below 2^-8 of its norm. A part of a cut tile is a float32 vector and its
logarithm, whose rounding (2^-24 of a score) is within the 2e-5 that exponents and powers have there. The turn: 2^-21 of the
pair's magnitudes and one rounding, as in the tests of the rotary positions."""
import numpy as np
import pytest
import torch

from helpers import have_gpu
from oracle.rotary import frequencies, rotary
from oracle.windowed import paged

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(int).tolist()


def _np(t):
    return t.double().cpu().numpy()


def compare(o, lse, ref, norm=True):
    eo, el, mass, size = ref
    g = _np(o)
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
        gl = _np(lse)
        lin = ~np.isnan(el)
        assert np.array_equal(np.isneginf(gl[lin]), np.isneginf(el[lin]))
        fin = np.isfinite(el)
        assert (np.abs(gl[fin] - el[fin]) <= (np.nan_to_num(size) * 4e-5 + 2e-5 + np.abs(np.where(fin, el, 0)) * 2.0 ** -22)[fin]).all()


class Cache:
    """A pool of NaN with pages for the given lengths in a shuffled order, NaN behind each sequence's last key too."""

    def __init__(self, lens, page, Hkv, D, seed=0, spare=3, wide=2, head_major=False):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        used = [-(-n // page) for n in lens]
        self.pages, self.page = sum(used) + spare, page
        order = rng.permutation(self.pages)
        cols = max(used + [0]) + wide
        self.table = np.full((len(lens), cols), -1)
        at = 0
        shape = (self.pages, Hkv, page, D) if head_major else (self.pages, page, Hkv, D)
        self.k, self.v = (torch.full(shape, float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
        if head_major:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        for b, (n, u) in enumerate(zip(lens, used)):
            self.table[b, :u] = order[at : at + u]
            at += u
            if n:
                j = torch.arange(n, device="cuda")
                entry = torch.tensor(self.table[b], device="cuda")[j // page]
                for t in (self.k, self.v):
                    t[entry, j % page] = torch.randn((n, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        self.dev = _i32(self.table.tolist()).view(len(lens), cols)

    def expect(self, q, lens, cu, **kw):
        return paged(_np(q), _np(self.k), _np(self.v), self.table.tolist(), lens, cu, **kw)


def _run(ss, lq, lens, Hq, Hkv, D, page, window=0, sinks=0, causal=True, seed=0, cu=True, head_major=False, hide=()):
    c = Cache(lens, page, Hkv, D, seed, head_major=head_major)
    for b, i in hide:
        c.table[b, i] = -1 if i % 2 else c.pages + 5
    c.dev = _i32(c.table.tolist()).view(c.table.shape)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn((sum(lq), Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    lse = torch.full((Hq, sum(lq)), 7.0, device="cuda")
    o = ss.attn_paged(q, c.k, c.v, c.dev, _i32(lens), cu_q=_i32(_cum(lq)) if cu else None, causal=causal, window=window or None,
                      sinks=sinks, lse=lse)
    compare(o, lse, c.expect(q, lens, _cum(lq), causal=causal, window=window, sinks=sinks))
    return c, q, o, lse


@pytest.mark.parametrize("page", [1, 3, 16, 24, 32, 64, 100])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 128), (7, 1, 64), (6, 2, 72), (33, 1, 32)])
@pytest.mark.parametrize("lens", [[1], [0, 5, 32, 33, 64, 0, 300], [777, 1, 2, 2049]], ids=str)
def test_single_tokens(ss, page, Hq, Hkv, D, lens):
    _run(ss, [1] * len(lens), lens, Hq, Hkv, D, page, seed=page)
    _run(ss, [1] * len(lens), lens, Hq, Hkv, D, page, seed=page, cu=False)


@pytest.mark.parametrize("D", [8, 16, 24, 40, 56, 64, 80, 96, 120, 128])
def test_head_sizes(ss, D):
    _run(ss, [2, 1, 5], [70, 200, 3], 4, 2, D, 16, seed=D)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lens", [([5], [5]), ([5], [3]), ([40], [41]), ([3, 0, 9, 1], [100, 7, 4, 0]), ([70, 33], [700, 33]),
                                     ([129], [1000])], ids=str)
@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 1, 128, 16), (5, 5, 64, 10), (64, 2, 128, 32)])
def test_chunks(ss, lq, lens, causal, Hq, Hkv, D, page):
    _run(ss, lq, lens, Hq, Hkv, D, page, causal=causal, seed=len(lq))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (31, 0), (32, 4), (33, 40), (64, 64), (100, 1000), (5000, 2)])
@pytest.mark.parametrize("lq,lens", [([1, 1, 1], [300, 64, 5]), ([6, 1, 40], [400, 0, 90]), ([3], [2000])], ids=str)
@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 1, 128, 16), (6, 3, 64, 40)])
def test_windows(ss, window, sinks, lq, lens, Hq, Hkv, D, page):
    """Pages that no row sees are given back: their entries name no page, and the pool's NaN there is not met."""
    hide = [(b, i) for b, (a, n) in enumerate(zip(lq, lens))
            for i in range(-(-sinks // page), max(max(n - a, 0) - window + 1, 0) // page)]
    _run(ss, lq, lens, Hq, Hkv, D, page, window, sinks, seed=window, hide=hide)


def test_entries_that_name_no_page(ss):
    """Their keys are seen by no row: in the middle of what a row sees, at both ends, all of them."""
    _run(ss, [1, 3, 1, 2], [200, 200, 90, 33], 4, 2, 128, 16, hide=[(0, 3), (0, 4), (1, 0), (1, 12), (2, 5), (2, 0), (3, 0), (3, 1), (3, 2)])
    _run(ss, [1, 2], [5000, 4000], 4, 2, 64, 16, hide=[(0, i) for i in range(0, 300, 7)] + [(1, i) for i in range(40, 250)])


@pytest.mark.parametrize("lens", [[40000], [9000, 17, 0, 20000, 1, 8000], [130] * 150, [2000 + 37 * i for i in range(40)],
                                  [(i * 7919) % 700 for i in range(300)]], ids=lambda v: f"{len(v)}-{v[0]}")
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (2, 1, 64)])
def test_runs_cut_anywhere(ss, lens, Hq, Hkv, D):
    """Sequences from one cut into hundreds of parts to hundreds in one run; the same call twice gives the same bits."""
    c, q, o, lse = _run(ss, [1] * len(lens), lens, Hq, Hkv, D, 16, seed=len(lens))
    lse2 = torch.empty_like(lse)
    o2 = ss.attn_paged(q, c.k, c.v, c.dev, _i32(lens), lse=lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [64, 128])
def test_many_calls_give_the_same_bits(ss, D):
    """Chunks whose tiles end inside a unit, cut into parts: loads of very different latency beside each other."""
    c = Cache([1000, 777], 32, 2, D, 1)
    q = torch.randn((129 + 50, 64, D), device="cuda").to(torch.bfloat16)
    cu, n = _i32([0, 129, 179]), _i32([1000, 777])
    first = ss.attn_paged(q, c.k, c.v, c.dev, n, cu_q=cu)
    compare(first, None, c.expect(q, [1000, 777], [0, 129, 179]))
    for _ in range(100):
        assert torch.equal(ss.attn_paged(q, c.k, c.v, c.dev, n, cu_q=cu), first)


def test_head_major_pages_and_strided_rows(ss):
    """Pages with the heads outside the keys, keys and values side by side in one pool, query and output rows inside wider ones."""
    _run(ss, [2, 1], [333, 40], 4, 2, 64, 16, head_major=True)
    c = Cache([300, 77], 16, 2, 64, 9)
    both = torch.stack((c.k, c.v), 1)  # [pages, 2, page, heads, values]
    wide = torch.randn((2, 9, 64), device="cuda").to(torch.bfloat16)
    out = torch.full((2, 11, 72), 3.0, device="cuda", dtype=torch.bfloat16)
    o = ss.attn_paged(wide[:, 2:6], both[:, 0], both[:, 1], c.dev, _i32([300, 77]), out=out[:, 1:5, :64])
    compare(o, None, c.expect(wide[:, 2:6], [300, 77], [0, 1, 2]))
    rest = out.clone()
    rest[:, 1:5, :64] = 3.0
    assert (rest == 3.0).all()


def test_rows_in_no_sequence_stay(ss):
    c = Cache([50, 60], 16, 1, 64, 2)
    q = torch.randn((9, 2, 64), device="cuda").to(torch.bfloat16)
    out, lse = torch.full_like(q, 5.0), torch.full((2, 9), 6.0, device="cuda")
    ss.attn_paged(q, c.k, c.v, c.dev, _i32([50, 60]), cu_q=_i32([2, 4, 7]), out=out, lse=lse)
    compare(out[2:7], lse[:, 2:7], c.expect(q[2:7], [50, 60], [0, 2, 5]))
    assert (out[:2] == 5).all() and (out[7:] == 5).all() and (lse[:, :2] == 6).all() and (lse[:, 7:] == 6).all()


def test_lengths_beyond_the_table_are_clamped(ss):
    c = Cache([64, 64], 16, 1, 64, 3, wide=0)
    q = torch.randn((2, 2, 64), device="cuda").to(torch.bfloat16)
    o = ss.attn_paged(q, c.k, c.v, c.dev, _i32([1 << 30, -5]))
    compare(o, None, c.expect(q, [64, 0], [0, 1, 2]))


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
@pytest.mark.parametrize("lens,Hq,Hkv,D", [([90], 4, 1, 128), ([4000], 40, 1, 64)])
def test_infinities_and_nan_reach_the_rows_that_see_them(ss, window, sinks, lens, Hq, Hkv, D):
    lq, lk = 6, lens[0]
    c = Cache(lens, 16, Hkv, D, 4)
    q = torch.randn((lq, Hq, D), device="cuda").to(torch.bfloat16)
    args = dict(cu_q=_i32([0, lq]), window=window or None, sinks=sinks)
    clean = ss.attn_paged(q, c.k, c.v, c.dev, _i32(lens), **args)
    assert clean.isfinite().all()
    p = torch.arange(lq, device="cuda") + lk - lq
    for j in (lk - 1, lk - 3, lk - lq, lk - 21, lk - 22, 2):
        rows = p >= j
        if window:
            rows &= (p - window < j) | (j < sinks)
        entry, at = int(c.table[0, j // 16]), j % 16
        v = c.v.clone()
        v[entry, at, :, 1], v[entry, at, :, 3] = float("nan"), float("inf")
        o = ss.attn_paged(q, c.k, v, c.dev, _i32(lens), **args)
        assert torch.equal(o[~rows], clean[~rows])
        other = [i for i in range(D) if i not in (1, 3)]
        assert torch.equal(o[:, :, other], clean[:, :, other])
        assert o[rows][:, :, 1].isnan().all() and (o[rows][:, :, 3] == float("inf")).all()
        k = c.k.clone()
        k[entry, at, :, 2] = float("nan")
        o = ss.attn_paged(q, k, c.v, c.dev, _i32(lens), **args)
        assert torch.equal(o[~rows], clean[~rows]) and o[rows].isnan().all()


def test_scores_of_any_size(ss):
    """Far apart scores: a row is the value of its largest one."""
    D, lk = 64, 3000
    c = Cache([lk], 16, 1, D, 5)
    for top in (20.0, 60.0, 110.0):
        q = torch.zeros((2, 2, D), device="cuda", dtype=torch.bfloat16)
        q[..., 0] = 2.0 ** top
        k = torch.zeros_like(c.k)
        best = torch.randint(0, lk - 2, (1,)).item()
        k[..., 0] = -1.0
        k[int(c.table[0, best // 16]), best % 16, :, 0] = 1.0
        v = torch.nan_to_num(c.v)
        o = ss.attn_paged(q, k, v, c.dev, _i32([lk]), cu_q=_i32([0, 2]), scale=1.0)
        assert torch.equal(o, v[int(c.table[0, best // 16]), best % 16].expand(2, 2, D))


def test_a_cache_beyond_32_bit_offsets(ss):
    Hkv, D, page = 8, 128, 1024
    pages = 4500  # 4.7e9 values an operand
    k = torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = [[4499, 0, 2100], [2047, 4400, 2048]]
    lens = [2500, 3000]
    small_k, small_v = (torch.randn((6, page, Hkv, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    for i, e in enumerate(sum(table, [])):
        k[e], v[e] = small_k[i], small_v[i]
    q = torch.randn((2, 16, D), device="cuda").to(torch.bfloat16)
    o = ss.attn_paged(q, k, v, _i32(table), _i32(lens))
    o2 = ss.attn_paged(q, small_k, small_v, _i32([[0, 1, 2], [3, 4, 5]]), _i32(lens))
    assert torch.equal(o, o2)
    compare(o, None, paged(_np(q), _np(small_k), _np(small_v), [[0, 1, 2], [3, 4, 5]], lens, [0, 1, 2]))
    kn, vn = (torch.randn((2, Hkv, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    ss.paged_store(kn, vn, _i32([2400, 1030]), k, v, _i32(table))
    assert torch.equal(k[2100, 2400 - 2048], kn[0]) and torch.equal(v[4400, 6], vn[1])


# ---- the write ---------------------------------------------------------------------------------------------------------


def _store(ss, lq, at, Hq, Hkv, D, page, rot, layout, seed=0, mscale=1.0, view=None, cu=True, in_place=False):
    """lq tokens of each sequence behind at[b] keys; everything that is not a place of one of them must stay."""
    T, lens = sum(lq), [a + n for a, n in zip(at, lq)]
    c = Cache(lens, page, Hkv, D, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    q, k, v = (torch.randn((T, H, D), generator=g, device="cuda").to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    if view:
        q, k, v = (view(t) for t in (q, k, v))
    pos = [a + i for a, n in zip(at, lq) for i in range(n)]
    seq = [b for b, n in enumerate(lq) for _ in range(n)]
    steps, _ = ss.rotary_steps(rot, 10000.0)
    freq, _ = frequencies(rot, 10000.0)
    before = [_np(t) for t in (q, k, v)]
    ek, ev = _np(c.k), _np(c.v)
    got = ss.paged_store(k, v, _i32(pos), c.k, c.v, c.dev, cu=_i32(_cum(lq)) if cu else None, q=q, steps=steps, layout=layout,
                         mscale=mscale, q_out=q if in_place else None)

    def turned(x):
        n = rot // 2
        exp = rotary(x, np.array(pos), freq, layout, mscale)
        ia, ib = (np.arange(n), np.arange(n) + n) if layout == "half" else (2 * np.arange(n), 2 * np.arange(n) + 1)
        size = np.zeros_like(x)
        size[..., ia] = size[..., ib] = (np.abs(x[..., ia]) + np.abs(x[..., ib])) * abs(mscale)
        return exp, 2.0 ** -21 * size + 2.0 ** -8 * (np.abs(exp) + 2.0 ** -21 * size) * (size > 0)

    eq, tol = turned(before[0])
    assert (np.abs(_np(got) - eq) <= tol).all()
    xk, tk = turned(before[1])
    hit = np.zeros(ek.shape[:2], bool)
    gk, gv = _np(c.k), _np(c.v)
    for t, (b, p) in enumerate(zip(seq, pos)):
        e, i = c.table[b, p // page], p % page
        hit[e, i] = True
        assert (np.abs(gk[e, i] - xk[t]) <= tk[t]).all() and np.array_equal(gv[e, i], before[2][t])
    assert np.array_equal(gk[~hit], ek[~hit], equal_nan=True) and np.array_equal(gv[~hit], ev[~hit], equal_nan=True)
    if in_place:
        assert got.data_ptr() == q.data_ptr()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("Hq,Hkv,D,rot", [(4, 1, 128, 128), (28, 4, 128, 64), (3, 3, 80, 22), (2, 2, 64, 16), (8, 1, 256, 256), (1, 1, 8, 2)])
@pytest.mark.parametrize("lq,at,page", [([1], [0], 16), ([3, 1, 50], [5, 0, 77], 16), ([1, 1, 1, 1], [15, 16, 100, 0], 24),
                                        ([300, 0, 7], [0, 4, 1000], 1)], ids=str)
def test_store(ss, layout, Hq, Hkv, D, rot, lq, at, page):
    _store(ss, lq, at, Hq, Hkv, D, page, rot, layout, seed=D)
    if all(n == 1 for n in lq):
        _store(ss, lq, at, Hq, Hkv, D, page, rot, layout, seed=D, cu=False, in_place=True, mscale=1.3)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_store_of_rows_off_16_bytes(ss, layout):
    def view(t):
        wide = torch.zeros((t.shape[0], t.shape[1], t.shape[2] + 3), dtype=t.dtype, device="cuda")
        wide[:, :, 1 : 1 + t.shape[2]] = t
        return wide[:, :, 1 : 1 + t.shape[2]]
    _store(ss, [9, 4], [3, 40], 6, 2, 64, 16, 64, layout, view=view)
    _store(ss, [9, 4], [3, 40], 6, 2, 64, 16, 20, layout, view=view, in_place=True)


def test_store_of_a_long_prompt(ss):
    _store(ss, [4000, 1, 2500], [0, 900, 333], 8, 2, 128, 64, 128, "half")


def test_store_without_queries_or_turns(ss):
    c = Cache([40, 3], 16, 2, 64, 1)
    k, v = (torch.randn((2, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    assert ss.paged_store(k, v, _i32([17, 2]), c.k, c.v, c.dev) is None
    for b, p in ((0, 17), (1, 2)):
        e = int(c.table[b, p // 16])
        assert torch.equal(c.k[e, p % 16], k[b]) and torch.equal(c.v[e, p % 16], v[b])


def test_store_leaves_alone_what_has_no_place(ss):
    """Tokens of no sequence, places before and behind the table, entries that name no page."""
    c = Cache([40, 40], 16, 1, 64, 1, wide=0)
    c.table[1, 1] = -7
    c.table[1, 2] = c.pages
    c.dev = _i32(c.table.tolist())
    T = 8
    q, k, v = (torch.randn((T, H, 64), device="cuda").to(torch.bfloat16) for H in (2, 1, 1))
    out = torch.full_like(q, 9.0)
    steps, _ = ss.rotary_steps(64)
    freq, _ = frequencies(64)
    pos = [3, -1, 48, 1 << 30, 20, 33, 7, 8]
    ek, ev = c.k.clone(), c.v.clone()
    ss.paged_store(k, v, _i32(pos), c.k, c.v, c.dev, cu=_i32([1, 4, 7]), q=q, steps=steps, q_out=out)
    e = int(c.table[1, 0])
    assert torch.equal(c.v[e, 7], v[6])
    ek[e, 7], ev[e, 7] = c.k[e, 7], c.v[e, 7]
    assert torch.equal(c.k.view(torch.int16), ek.view(torch.int16)) and torch.equal(c.v.view(torch.int16), ev.view(torch.int16))
    exp = rotary(_np(q), np.array(pos), freq)
    assert (out[0] == 9).all() and (out[7] == 9).all()
    near = np.abs(_np(out) - exp)[1:7]
    assert (near <= 2.0 ** -8 * np.abs(exp[1:7]) + 2.0 ** -20 * np.abs(_np(q)).max()).all()


# ---- together ------------------------------------------------------------------------------------------------------------


def test_decode_steps_captured_and_replayed(ss):
    """Write and attention of one token each, captured once: the replays read positions, lengths, tables and inputs anew. The
    lengths grow from empty to cut tiles; eager calls and synchronisations stand between the replays."""
    B, Hq, Hkv, D, page, cols = 3, 8, 2, 64, 16, 200
    steps, _ = ss.rotary_steps(D)
    pool = [torch.full((B * cols, page, Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    for t in pool:
        t.copy_(torch.randn(t.shape, device="cuda"))
    table = torch.randperm(B * cols, device="cuda").to(torch.int32).view(B, cols)
    q, k, v = (torch.zeros((B, H, D), device="cuda", dtype=torch.bfloat16) for H in (Hq, Hkv, Hkv))
    pos, n = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        turned = ss.paged_store(k, v, pos, pool[0], pool[1], table, q=q, steps=steps)
        return ss.attn_paged(turned, pool[0], pool[1], table, n), ss.attn_paged(turned, pool[0], pool[1], table, n, window=100, sinks=4)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        full, near = step()
    for at in ([0, 1, 2], [15, 16, 3000], [500, 31, 3199], [0, 0, 0], [3100, 3000, 2900]):
        pos.copy_(_i32(at))
        n.copy_(pos + 1)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = full.clone(), near.clone()
        exp = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], exp[0]) and torch.equal(got[1], exp[1])
        turned = ss.rotary(q, pos, steps)
        host = [_np(t) for t in pool]
        for o, w, s in ((full, 0, 0), (near, 100, 4)):
            compare(o, None, paged(_np(turned), *host, table.tolist(), [a + 1 for a in at], [0, 1, 2, 3], window=w, sinks=s))


def test_two_streams_with_workspaces_of_their_own(ss):
    lens = [5000, 3000]
    c = Cache(lens, 16, 2, 128, 8)
    qs = [torch.randn((2, 8, 128), device="cuda").to(torch.bfloat16) for _ in range(2)]
    need = ss.attn_paged_workspace_bytes(2, c.table.shape[1] * 16, 2, 8, 2, 128)
    assert need > 0
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2)]
    n = _i32(lens)
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, w, o in zip(streams, qs, spaces, outs):
            with torch.cuda.stream(s):
                ss.attn_paged(q, c.k, c.v, c.dev, n, workspace=w, out=o)
    torch.cuda.synchronize()
    for q, o in zip(qs, outs):
        compare(o, None, c.expect(q, lens, [0, 1, 2]))
