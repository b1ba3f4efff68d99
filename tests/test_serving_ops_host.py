"""Host side of the norm, the paged cache's calls and the windowed attention (no GPU needed): what they refuse, and that
nothing is launched for empty problems."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "structured_sparse_quantized_amd", "libss.so")),
                                reason="libss.so not built")
FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)  # never dereferenced: validation fails first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


def _statuses(call, good, cases):
    """`call(**good)` with one or two arguments changed each: the status it must return."""
    for change, status in cases:
        assert call(**{**good, **change}) == status, change


def test_norm_refusals(ss):
    good = dict(X=FAKE, xt=ss.SS_BF16, M=4, K=64, ldx=64, res=FAKE, ldr=64, sum=FAKE, lds=64, w=FAKE, wt=ss.SS_BF16, eps=1e-5, n=2,
                yt=ss.SS_I8, Y=ctypes.c_void_p(1 << 21), ldy=256, sx=FAKE)
    call = lambda **a: ss.lib.ss_rmsnorm_act(*a.values(), None)  # noqa: E731
    _statuses(call, good, [
        (dict(n=1), ss.SS_ERR_PATTERN), (dict(n=9), ss.SS_ERR_PATTERN), (dict(xt=ss.SS_I8), ss.SS_ERR_DTYPE),
        (dict(yt=ss.SS_I32), ss.SS_ERR_DTYPE), (dict(yt=ss.SS_F32), ss.SS_ERR_DTYPE), (dict(xt=ss.SS_F32), ss.SS_ERR_DTYPE),
        (dict(wt=ss.SS_I8), ss.SS_ERR_DTYPE), (dict(yt=ss.SS_BF16, n=3, sx=None), ss.SS_ERR_PATTERN),
        (dict(yt=ss.SS_BF16), ss.SS_ERR_DTYPE), (dict(eps=-1.0), ss.SS_ERR_SHAPE), (dict(eps=NAN), ss.SS_ERR_SHAPE),
        (dict(eps=INF), ss.SS_ERR_SHAPE), (dict(M=-1), ss.SS_ERR_SHAPE), (dict(K=-1), ss.SS_ERR_SHAPE), (dict(M=1 << 31), ss.SS_ERR_SHAPE),
        (dict(X=None), ss.SS_ERR_NULL), (dict(X=ODD), ss.SS_ERR_ALIGN), (dict(ldx=63), ss.SS_ERR_SHAPE), (dict(ldx=68), ss.SS_ERR_ALIGN),
        (dict(res=ODD), ss.SS_ERR_ALIGN), (dict(ldr=60), ss.SS_ERR_SHAPE), (dict(sum=None), ss.SS_ERR_NULL),
        (dict(res=None), ss.SS_ERR_UNSUPPORTED), (dict(lds=72), ss.SS_ERR_SHAPE), (dict(Y=None), ss.SS_ERR_NULL),
        (dict(ldy=64), ss.SS_ERR_SHAPE), (dict(Y=FAKE), ss.SS_ERR_UNSUPPORTED), (dict(sx=None), ss.SS_ERR_NULL),
        (dict(w=ODD), ss.SS_ERR_ALIGN), (dict(M=0, X=None), ss.SS_OK), (dict(K=0, X=None), ss.SS_OK)])


def test_window_refusals(ss):
    good = dict(q=FAKE, sqt=512, sqh=128, k=FAKE, skt=128, skh=128, v=FAKE, svt=128, svh=128, o=FAKE, sot=512, soh=128, lse=None, Tq=9,
                Tk=50, B=1, Hq=4, Hkv=1, D=128, cu_q=None, cu_k=None, k_len=None, scale=0.1, causal=1, window=5, sinks=1, ws=None,
                bytes=0)
    call = lambda **a: ss.lib.ss_attn_window(*a.values(), None)  # noqa: E731
    _statuses(call, good, [
        (dict(window=-1), ss.SS_ERR_SHAPE), (dict(sinks=-1), ss.SS_ERR_SHAPE), (dict(causal=0), ss.SS_ERR_UNSUPPORTED),
        (dict(D=12), ss.SS_ERR_UNSUPPORTED), (dict(Hkv=3), ss.SS_ERR_SHAPE), (dict(scale=0.0), ss.SS_ERR_SHAPE),
        (dict(q=ODD), ss.SS_ERR_ALIGN), (dict(sot=100), ss.SS_ERR_ALIGN), (dict(B=2), ss.SS_ERR_NULL), (dict(Tq=0), ss.SS_OK),
        (dict(B=-1), ss.SS_ERR_SHAPE)])
    need = ss.attn_window_workspace_bytes(1, 50000, 1, 8, 2, 64, 4096, 4)
    assert need > 0
    many = dict(good, Tq=1, Tk=50000, Hq=8, Hkv=2, D=64, window=4096)
    assert call(**many) == ss.SS_ERR_NULL and call(**{**many, "ws": ODD, "bytes": need}) == ss.SS_ERR_ALIGN
    assert call(**{**many, "ws": FAKE, "bytes": need - 1}) == ss.SS_ERR_SHAPE
    # a window beside few keys, and no window at all
    assert ss.attn_window_workspace_bytes(1, 50000, 1, 8, 2, 64, 60, 0) == 0
    assert ss.attn_window_workspace_bytes(1, 50000, 1, 8, 2, 64, 0, 9) == ss.attn_workspace_bytes(1, 50000, 1, 8, 2, 64)
    assert ss.attn_window_workspace_bytes(1, 50000, 1, 8, 2, 64, -1, 0) == -1


def _kv(ss, **change):
    f = dict(k=1 << 20, v=1 << 20, pages=10, page=16, skp=16 * 256, skt=256, skh=128, svp=16 * 256, svt=256, svh=128, table=1 << 20,
             table_cols=6, table_ld=6)
    return ctypes.byref(ss.PagedKV(**{**f, **change}))


CACHES = [(dict(k=None), "SS_ERR_NULL"), (dict(v=(1 << 20) + 8), "SS_ERR_ALIGN"), (dict(page=0), "SS_ERR_SHAPE"), (dict(pages=-1), "SS_ERR_SHAPE"),
          (dict(skp=16 * 256 + 4), "SS_ERR_ALIGN"), (dict(skt=-256), "SS_ERR_SHAPE"), (dict(svh=124), "SS_ERR_ALIGN"),
          (dict(skp=1 << 33), "SS_ERR_UNSUPPORTED"), (dict(svt=1 << 24), "SS_ERR_UNSUPPORTED"), (dict(table=None), "SS_ERR_NULL"),
          (dict(table=(1 << 20) + 2), "SS_ERR_ALIGN"), (dict(table_ld=5), "SS_ERR_SHAPE"), (dict(table_cols=-1), "SS_ERR_SHAPE"),
          (dict(pages=1 << 32), "SS_ERR_SHAPE")]


def test_paged_attention_refusals(ss):
    wide = _kv(ss, table_cols=600, table_ld=600)  # (room that asks for a workspace)
    good = dict(q=FAKE, sqt=512, sqh=128, kv=wide, o=FAKE, sot=512, soh=128, lse=None, Tq=3, B=3, Hq=4, Hkv=2, D=128, cu_q=None,
                k_len=FAKE, scale=0.1, causal=1, window=0, sinks=0, ws=FAKE, bytes=1 << 40)
    call = lambda **a: ss.lib.ss_attn_paged(*a.values(), None)  # noqa: E731
    _statuses(call, good, [
        (dict(kv=None), ss.SS_ERR_NULL), (dict(q=None), ss.SS_ERR_NULL), (dict(q=ODD), ss.SS_ERR_ALIGN), (dict(o=None), ss.SS_ERR_NULL),
        (dict(soh=120), ss.SS_ERR_SHAPE), (dict(sqt=-512), ss.SS_ERR_SHAPE), (dict(k_len=None), ss.SS_ERR_NULL), (dict(Hkv=3), ss.SS_ERR_SHAPE),
        (dict(D=136), ss.SS_ERR_UNSUPPORTED), (dict(D=4), ss.SS_ERR_UNSUPPORTED), (dict(scale=NAN), ss.SS_ERR_SHAPE),
        (dict(window=3, causal=0), ss.SS_ERR_UNSUPPORTED), (dict(window=-3), ss.SS_ERR_SHAPE), (dict(Tq=5), ss.SS_ERR_NULL),
        (dict(ws=None), ss.SS_ERR_NULL), (dict(ws=ODD), ss.SS_ERR_ALIGN), (dict(bytes=100), ss.SS_ERR_SHAPE), (dict(bytes=-1), ss.SS_ERR_SHAPE),
        (dict(k_len=ctypes.c_void_p(2)), ss.SS_ERR_ALIGN), (dict(Tq=0, q=None), ss.SS_OK), (dict(B=0, q=None), ss.SS_OK),
        (dict(Tq=1 << 27, B=1 << 27, Hq=64, Hkv=64, D=8), ss.SS_ERR_SHAPE)])
    for change, status in CACHES:
        assert call(**{**good, "kv": _kv(ss, **change)}) == getattr(ss, status), change
    assert ss.attn_paged_workspace_bytes(3, 96, 3, 4, 2, 128) == 0 and ss.attn_paged_workspace_bytes(3, 9600, 3, 4, 2, 128) > 0
    assert ss.attn_paged_workspace_bytes(3, -1, 3, 4, 2, 128) == -1 and ss.attn_paged_workspace_bytes(3, 96, 3, 4, 3, 128) == -1


def test_store_refusals(ss):
    good = dict(q=FAKE, sqt=512, sqh=128, k=FAKE, skt=256, skh=128, v=FAKE, svt=256, svh=128, T=3, B=3, Hq=4, Hkv=2, D=128, pos=FAKE,
                cu=None, steps=FAKE, rot=128, layout=0, mscale=1.0, qo=FAKE, sot=512, soh=128, kv=_kv(ss))
    call = lambda **a: ss.lib.ss_paged_store(*a.values(), None)  # noqa: E731
    _statuses(call, good, [
        (dict(kv=None), ss.SS_ERR_NULL), (dict(q=None), ss.SS_ERR_NULL), (dict(k=None), ss.SS_ERR_NULL), (dict(v=ctypes.c_void_p(3)), ss.SS_ERR_ALIGN),
        (dict(qo=None), ss.SS_ERR_NULL), (dict(pos=None), ss.SS_ERR_NULL), (dict(steps=None), ss.SS_ERR_NULL), (dict(steps=ctypes.c_void_p(4)), ss.SS_ERR_ALIGN),
        (dict(rot=3), ss.SS_ERR_SHAPE), (dict(rot=130), ss.SS_ERR_SHAPE), (dict(rot=-2), ss.SS_ERR_SHAPE), (dict(rot=0), ss.SS_ERR_UNSUPPORTED),
        (dict(layout=2), ss.SS_ERR_UNSUPPORTED), (dict(mscale=INF), ss.SS_ERR_SHAPE), (dict(B=2), ss.SS_ERR_NULL), (dict(D=20), ss.SS_ERR_UNSUPPORTED),
        (dict(skt=-1), ss.SS_ERR_SHAPE), (dict(soh=64), ss.SS_ERR_SHAPE), (dict(sot=640), ss.SS_ERR_SHAPE), (dict(T=-1), ss.SS_ERR_SHAPE),
        (dict(T=0, k=None), ss.SS_OK), (dict(Hkv=0, k=None), ss.SS_ERR_SHAPE), (dict(Hkv=0, Hq=0, k=None), ss.SS_OK)])
    for change, status in CACHES + [(dict(skh=64), "SS_ERR_SHAPE"), (dict(svt=0), "SS_ERR_SHAPE"), (dict(skp=0), "SS_ERR_SHAPE")]:
        assert call(**{**good, "kv": _kv(ss, **change)}) == getattr(ss, status), change


def _raises(ss, status, f):
    with pytest.raises(ss.SSError) as e:
        f()
    assert e.value.status == status, e.value


def test_the_binding_refuses_before_it_looks_for_a_gpu(ss):
    """Sizes and types of host tensors: every mistake is named; a call without one ends at the tensors' device."""
    bf, i32 = torch.bfloat16, torch.int32
    x, w = torch.zeros((4, 64), dtype=bf), torch.zeros(64, dtype=bf)
    n = lambda *a, **k: (lambda: ss.rmsnorm_act(*a, **k))  # noqa: E731
    for status, f in [(ss.SS_ERR_UNSUPPORTED, n(x, w)), (ss.SS_ERR_SHAPE, n(x[0], w)), (ss.SS_ERR_SHAPE, n(x, w[:60])), (ss.SS_ERR_DTYPE, n(x.half(), w)),
                      (ss.SS_ERR_DTYPE, n(x, w.half())), (ss.SS_ERR_DTYPE, n(x, w, residual=x.float())), (ss.SS_ERR_SHAPE, n(x, w, residual=x[:3])),
                      (ss.SS_ERR_UNSUPPORTED, n(x, w, sum_out=x)), (ss.SS_ERR_SHAPE, n(x, w, residual=x, sum_out=x[:, :60])),
                      (ss.SS_ERR_PATTERN, n(x, w, n=1, y_dtype="i8")), (ss.SS_ERR_DTYPE, n(x, w, y_dtype="f32")),
                      (ss.SS_ERR_SHAPE, n(x, w, y_dtype="i8", out=torch.zeros((4, 64), dtype=torch.int8))),
                      (ss.SS_ERR_DTYPE, n(x, w, y_dtype="i8", out=x)), (ss.SS_ERR_DTYPE, n(x, w, scale_out=torch.zeros(4))),
                      (ss.SS_ERR_SHAPE, n(x.t(), w[:4])), (ss.SS_ERR_SHAPE, n(x, w, y_dtype="i8", scale_out=torch.zeros(3)))]:
        _raises(ss, status, f)

    q, kp, t, ln = torch.zeros((3, 4, 64), dtype=bf), torch.zeros((5, 16, 2, 64), dtype=bf), torch.zeros((3, 6), dtype=i32), torch.zeros(3, dtype=i32)
    p = lambda *a, **k: (lambda: ss.attn_paged(*a, **k))  # noqa: E731
    for status, f in [(ss.SS_ERR_UNSUPPORTED, p(q, kp, kp, t, ln)), (ss.SS_ERR_SHAPE, p(q, kp, kp[:4], t, ln)), (ss.SS_ERR_SHAPE, p(q, kp, kp, t[:2], ln)),
                      (ss.SS_ERR_SHAPE, p(q, kp[0], kp[0], t, ln)), (ss.SS_ERR_SHAPE, p(q[..., :32], kp, kp, t, ln)), (ss.SS_ERR_DTYPE, p(q, kp, kp.float(), t, ln)),
                      (ss.SS_ERR_DTYPE, p(q, kp, kp, t.long(), ln)), (ss.SS_ERR_DTYPE, p(q, kp, kp, t, ln.long())), (ss.SS_ERR_SHAPE, p(q, kp, kp, t, ln, cu_q=ln)),
                      (ss.SS_ERR_SHAPE, p(q, kp, kp, t, ln, window=0)), (ss.SS_ERR_SHAPE, p(q, kp, kp, t, ln, out=q[:2])), (ss.SS_ERR_SHAPE, p(q, kp, kp, t.t(), ln[:1])),
                      (ss.SS_ERR_SHAPE, p(q, kp, kp, t, ln, lse=torch.zeros((3, 4)))), (ss.SS_ERR_DTYPE, p(q.float(), kp, kp, t, ln))]:
        _raises(ss, status, f)

    k, pos, st = torch.zeros((3, 2, 64), dtype=bf), torch.zeros(3, dtype=i32), torch.zeros(32, dtype=torch.int64)
    s = lambda *a, **k: (lambda: ss.paged_store(*a, **k))  # noqa: E731
    for status, f in [(ss.SS_ERR_UNSUPPORTED, s(k, k, pos, kp, kp, t, q=q, steps=st)), (ss.SS_ERR_NULL, s(k, k, pos, kp, kp, t, q=q)),
                      (ss.SS_ERR_SHAPE, s(k, k[:2], pos, kp, kp, t)), (ss.SS_ERR_SHAPE, s(k, k, pos[:2], kp, kp, t)), (ss.SS_ERR_SHAPE, s(k, k, pos, kp, kp, t, q=q[:2], steps=st)),
                      (ss.SS_ERR_UNSUPPORTED, s(k, k, pos, kp, kp, t, q_out=q)), (ss.SS_ERR_SHAPE, s(k, k, pos, kp, kp, t, cu=pos)), (ss.SS_ERR_DTYPE, s(k, k, pos.long(), kp, kp, t)),
                      (ss.SS_ERR_UNSUPPORTED, s(k, k, pos, kp, kp, t, layout="quarter")), (ss.SS_ERR_SHAPE, s(k, k, pos, kp[..., :32], kp, t)),
                      (ss.SS_ERR_DTYPE, s(k, k.float(), pos, kp, kp, t)), (ss.SS_ERR_DTYPE, s(k, k, pos, kp, kp, t, q=q, steps=st.int()))]:
        _raises(ss, status, f)
    _raises(ss, ss.SS_ERR_SHAPE, lambda: ss.attn(q, q, q, window=-2))
    _raises(ss, ss.SS_ERR_SHAPE, lambda: ss.attn(q, q, q, window=4, sinks=-1))
    with pytest.raises(TypeError):
        ss.rmsnorm_act([1.0], w)
