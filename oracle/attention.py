"""Attention of packed sequences with grouped heads in float64, one query row at a time."""
import numpy as np


def attention(q, k, v, cu_q, cu_k, k_len=None, causal=True, scale=None):
    """q [Tq, Hq, D], k / v [Tk, Hkv, D] -> (o [Tq, Hq, D], lse [Hq, Tq], mass [Tq, Hq, D], size [Hq, Tq]). Rows of no
    sequence are NaN in all of them. mass = sum_j p_j |v_j| and size = max_j scale * sum_d |q_d k_jd| bound what
    rounding can do to a row."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    Tq, Hq, D = q.shape
    G = Hq // k.shape[1] if k.shape[1] else 1
    scale = D ** -0.5 if scale is None else scale
    o, mass = np.full((Tq, Hq, D), np.nan), np.full((Tq, Hq, D), np.nan)
    lse, size = np.full((Hq, Tq), np.nan), np.full((Hq, Tq), np.nan)
    for b in range(len(cu_q) - 1):
        lq, k0 = cu_q[b + 1] - cu_q[b], cu_k[b]
        lk = cu_k[b + 1] - k0
        if k_len is not None:
            lk = min(lk, k_len[b])
        for i in range(lq):
            n = min(max(i + lk - lq + 1, 0), lk) if causal else lk
            r = cu_q[b] + i
            for a in range(Hq):
                if n == 0:
                    o[r, a], mass[r, a], lse[a, r], size[a, r] = 0.0, 0.0, -np.inf, 0.0
                    continue
                kk, vv = k[k0 : k0 + n, a // G], v[k0 : k0 + n, a // G]
                s = scale * (kk @ q[r, a])
                e = np.exp(s - s.max())
                p = e / e.sum()
                o[r, a], mass[r, a] = p @ vv, p @ np.abs(vv)
                lse[a, r] = s.max() + np.log(e.sum())
                size[a, r] = scale * (np.abs(kk) @ np.abs(q[r, a])).max()
    return o, lse, mass, size
