"""Rotary positions in float64: frequencies with their scalings, and the turn of each pair."""
import math

import numpy as np


def frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=4.0):
    """(radians per position of each pair, factor on the turned values)."""
    out = []
    for i in range(rot_dim // 2):
        b = base
        if scaling == "ntk" and rot_dim > 2:
            b = base * factor ** (rot_dim / (rot_dim - 2))
        f = 1.0 / b ** (2.0 * i / rot_dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "smooth":
            turns = original * f / (2.0 * math.pi)
            if turns <= low:
                f = f / factor
            elif turns < high:
                w = (turns - low) / (high - low)
                f = w * f + (1.0 - w) * f / factor
        elif scaling == "yarn":
            def pair(turns):
                return rot_dim * math.log(original / (2.0 * math.pi * turns)) / (2.0 * math.log(base))
            first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot_dim - 1)
            w = (i - first) / max(last - first, 0.001)
            w = min(max(w, 0.0), 1.0)
            f = w * f / factor + (1.0 - w) * f
        out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def rotary(x, pos, freq, layout="half", mscale=1.0, inverse=False):
    """x [T, H, D] -> the same in float64, the first 2 len(freq) values of each head turned."""
    x = np.asarray(x, np.float64)
    n = len(freq)
    t = np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float64)[None, :]
    c, s = mscale * np.cos(t)[:, None, :], mscale * np.sin(t)[:, None, :]
    if inverse:
        s = -s
    y = x.copy()
    ia, ib = (np.arange(n), np.arange(n) + n) if layout == "half" else (2 * np.arange(n), 2 * np.arange(n) + 1)
    a, b = x[:, :, ia], x[:, :, ib]
    y[:, :, ia] = a * c - b * s
    y[:, :, ib] = b * c + a * s
    return y
