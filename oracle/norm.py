"""Root-mean-square norm of rows with the residual's addition, step by step as the library states it: the sum rounded to the
stream's type, the mean and the root in float64, two float32 products. What follows (bf16, or codes and lift) works on the row z."""
import numpy as np

from .quant import QMAX, e4m3_encode, f32_to_bf16_rne
from .slide import lift, lifted_k_alloc


def rmsnorm(x, w=None, eps=1e-6, residual=None, bf16=True):
    """x, residual [M, K] float32 values of the stream's type -> (z [M, K] float32, sum [M, K] float32)."""
    r = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        if residual is not None:
            r = (r + np.asarray(residual, np.float32)).astype(np.float32)
            if bf16:
                r = f32_to_bf16_rne(r)
        m = (r.astype(np.float64) ** 2).mean(1) + eps
        # a row of zeros without eps: 0; beyond float32: its largest number; of a NaN: NaN; of an infinity: 0
        rs = np.minimum(1.0 / np.sqrt(np.where(m == 0, 1.0, m)), np.float64(np.finfo(np.float32).max))
        rs = np.where(m == 0, 0.0, rs).astype(np.float32)
        z = (r * rs[:, None]).astype(np.float32)
        if w is not None:
            z = (z * np.asarray(w, np.float32)).astype(np.float32)
    return z, r


def codes(z, n, q):
    """The row's codes, with inv = fl32(fl32(1 / a) Q), lifted to K' and padded, and its scale fl32(a / Q). A row with a NaN
    or an infinity (a is one then) has codes of zero."""
    z = np.asarray(z, np.float32)
    a, Q = np.abs(z).max(1), np.float32(QMAX[q])
    some = (a > 0) & np.isfinite(a)
    one = np.where(some, a, np.float32(1)).astype(np.float32)
    t = (np.where(some[:, None], z, np.float32(0)) * ((np.float32(1) / one).astype(np.float32) * Q)[:, None]).astype(np.float32)
    c = np.clip(np.rint(t), -127, 127).astype(np.int8) if q == "i8" else e4m3_encode(np.clip(t, -448.0, 448.0))
    c[~some] = 0
    y = lift(c, n)
    out = np.zeros((z.shape[0], lifted_k_alloc(z.shape[1], n)), y.dtype)
    out[:, : y.shape[1]] = y
    return out, (a / Q).astype(np.float32)
