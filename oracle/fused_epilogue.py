"""What follows a linear layer: bias, activation, gate, residual; in float64, or step by step in float32."""
import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activate(z, act):
    z = np.asarray(z, np.float64)
    if act == "relu":
        return np.where(z > 0, z, 0.0)
    if act == "gelu":
        return z / 2 * (1 + _erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return z / 2 * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * np.where(z > 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
    return z


def epilogue(y, bias=None, act="none", gated=False, residual=None):
    """y [M, N] (the scaled product) in float64 -> [M, N] or, gated, [M, N / 2]."""
    z = np.asarray(y, np.float64)
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    v = activate(z[:, 0::2], act) * z[:, 1::2] if gated else activate(z, act)
    return v if residual is None else v + np.asarray(residual, np.float64)


def epilogue_f32(y, bias=None, relu=False, gated=False, residual=None):
    """The same for no activation or ReLU with every step rounded to float32, as the product does it."""
    z = np.asarray(y, np.float32)
    if bias is not None:
        z = z + np.asarray(bias, np.float32)
    a = np.maximum(z, np.float32(0)) if relu else z
    v = a[:, 0::2] * z[:, 1::2] if gated else a
    return v if residual is None else v + np.asarray(residual, np.float32)
