"""Attention of packed sequences under a sliding window with first tokens that stay visible, and over paged caches, in
float64."""
import numpy as np


def seen(lq, lk, causal=True, window=0, sinks=0):
    """[lq, lk]: which key a row sees."""
    p = np.arange(lq)[:, None] + lk - lq
    j = np.arange(lk)[None, :]
    if not causal:
        return np.ones((lq, lk), bool)
    see = j <= p
    if window:
        see = see & ((j > p - window) | (j < sinks))
    return see


def attend(q, k, v, see, scale=None):
    """One sequence: q [lq, Hq, D], k / v [lk, Hkv, D], see [lq, lk] -> (o, lse [Hq, lq], mass, size [Hq, lq]); rows that see
    nothing give zeros and -inf. mass = sum_j p_j |v_j|, size = max_j scale sum_d |q_d k_jd| over the seen keys."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    lq, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    o, mass = np.zeros((lq, Hq, D)), np.zeros((lq, Hq, D))
    lse, size = np.full((Hq, lq), -np.inf), np.zeros((Hq, lq))
    if k.shape[0] == 0:
        return o, lse, mass, size
    some = see.any(1)
    for a in range(Hq):
        kk, vv = np.where(see.any(0)[:, None], k[:, a // G], 0), np.where(see.any(0)[:, None], v[:, a // G], 0)
        s = np.where(see, scale * (q[:, a] @ kk.T), -np.inf)
        m = np.where(some, s.max(1), 0.0)
        e = np.exp(s - m[:, None])
        n = np.where(some, e.sum(1), 1.0)
        o[:, a], mass[:, a] = (e / n[:, None]) @ vv, (e / n[:, None]) @ np.abs(vv)
        lse[a] = np.where(some, m + np.log(n), -np.inf)
        size[a] = np.where(see, scale * (np.abs(q[:, a]) @ np.abs(kk).T), 0).max(1)
    return o, lse, mass, size


def packed(q, k, v, cu_q, cu_k, k_len=None, causal=True, window=0, sinks=0, scale=None):
    """All sequences of a call; rows of no sequence are NaN."""
    Tq, Hq, D = q.shape
    o, mass = np.full((Tq, Hq, D), np.nan), np.full((Tq, Hq, D), np.nan)
    lse, size = np.full((Hq, Tq), np.nan), np.full((Hq, Tq), np.nan)
    for b in range(len(cu_q) - 1):
        r, k0 = slice(cu_q[b], cu_q[b + 1]), cu_k[b]
        lk = cu_k[b + 1] - k0 if k_len is None else min(cu_k[b + 1] - k0, k_len[b])
        see = seen(cu_q[b + 1] - cu_q[b], lk, causal, window, sinks)
        o[r], lse[:, r], mass[r], size[:, r] = attend(q[r], k[k0 : k0 + lk], v[k0 : k0 + lk], see, scale)
    return o, lse, mass, size


def paged(q, k_pages, v_pages, table, k_len, cu_q, causal=True, window=0, sinks=0, scale=None):
    """The same over k_pages / v_pages [pages, page, Hkv, D]; keys whose entry names no page are seen by no row."""
    Tq, Hq, D = q.shape
    pages, page = k_pages.shape[:2]
    o, mass = np.full((Tq, Hq, D), np.nan), np.full((Tq, Hq, D), np.nan)
    lse, size = np.full((Hq, Tq), np.nan), np.full((Hq, Tq), np.nan)
    for b in range(len(cu_q) - 1):
        r = slice(cu_q[b], cu_q[b + 1])
        lk = max(min(k_len[b], len(table[b]) * page), 0)
        j = np.arange(lk)
        entry = np.asarray(table[b], np.int64)[j // page] if lk else np.zeros(0, np.int64)
        there = (entry >= 0) & (entry < pages)
        see = seen(cu_q[b + 1] - cu_q[b], lk, causal, window, sinks) & there[None, :]
        at = np.where(there, entry, 0)
        o[r], lse[:, r], mass[r], size[:, r] = attend(q[r], k_pages[at, j % page], v_pages[at, j % page], see, scale)
    return o, lse, mass, size
