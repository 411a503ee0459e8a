"""Plain fp64 forms of the 8-bit path and of the norm ahead of it: quantising
in blocks of 128, the product of what was quantised, layer norm and its
backward pass.  Test infrastructure only; written from the formulas in
include/flashsample.h.
"""

from dataclasses import dataclass

import numpy as np

BLOCK = 128
E4M3, E5M2 = "e4m3", "e5m2"
LARGEST = {E4M3: 448.0, E5M2: 57344.0}
_MANTISSA = {E4M3: 3, E5M2: 2}
_LEAST_EXPONENT = {E4M3: -6, E5M2: -14}


def round_fp8(v, fmt):
    """The nearest 8-bit values to v (fp64, |v| up to the largest), ties to
    even mantissas; NaN stays NaN."""
    v = np.asarray(v, np.float64)
    with np.errstate(all="ignore"):
        _, e = np.frexp(np.where(np.isfinite(v), v, 0.0))
        step = np.ldexp(1.0, np.maximum(e - 1, _LEAST_EXPONENT[fmt]) - _MANTISSA[fmt])
        return np.rint(v / step) * step


def _spread(scale, rows, cols, block_rows):
    return np.repeat(np.repeat(scale, block_rows, 0)[:rows], BLOCK, 1)[:, :cols]


@dataclass
class Quantised:
    q: np.ndarray        # fp64 values of the 8-bit elements [R, C]
    scale: np.ndarray    # fp64 [ceil(R / block_rows), ceil(C / 128)]
    value: np.ndarray    # q times its block's scale [R, C]


def quantise(x, block_rows=1, fmt=E4M3):
    """Scale, reciprocal and product are each rounded to fp32, as the header
    defines them (fp64 quotients of fp32 numbers round to the fp32 ones)."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    rb, cb = -(-R // block_rows), -(-C // BLOCK)
    size = np.zeros((rb * block_rows, cb * BLOCK))
    size[:R, :C] = np.where(np.isnan(x), 0.0, np.abs(x.astype(np.float64)))
    amax = size.reshape(rb, block_rows, cb, BLOCK).max((1, 3))
    with np.errstate(all="ignore"):
        scale = np.maximum((amax / LARGEST[fmt]).astype(np.float32), np.float32(2.0 ** -100))
        inverse = (1.0 / scale.astype(np.float64)).astype(np.float32)
        scaled = x.astype(np.float64) * _spread(inverse.astype(np.float64), R, C, block_rows)
        q = round_fp8(scaled.astype(np.float32).astype(np.float64), fmt)
        scale = scale.astype(np.float64)
        return Quantised(q, scale, q * _spread(scale, R, C, block_rows))


def product(a, b):
    """a bᵀ of two Quantised, and the sum of the magnitudes of its terms."""
    return a.value @ b.value.T, np.abs(a.value) @ np.abs(b.value).T


@dataclass
class Norm:
    mean: np.ndarray     # [n] (zeros with rms)
    rstd: np.ndarray     # [n]
    xh: np.ndarray       # [n, d]
    y: np.ndarray        # [n, d]


def layer_norm(x, weight=None, bias=None, eps=1e-5, rms=False):
    x = np.asarray(x, np.float64)
    d = x.shape[1]
    mean = np.zeros(len(x)) if rms else x.mean(1)
    centred = x - mean[:, None]
    rstd = 1.0 / np.sqrt((centred ** 2).sum(1) / d + eps)
    xh = centred * rstd[:, None]
    w = np.ones(d) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(d) if bias is None else np.asarray(bias, np.float64)
    return Norm(mean, rstd, xh, xh * w + b)


def layer_norm_gradients(g, norm, weight=None, rms=False):
    """(grad_x, grad_weight, grad_bias) for g = dL/dy."""
    g = np.asarray(g, np.float64)
    a = g if weight is None else g * np.asarray(weight, np.float64)
    gx = a - norm.xh * (a * norm.xh).mean(1, keepdims=True)
    if not rms:
        gx = gx - a.mean(1, keepdims=True)
    return gx * norm.rstd[:, None], (g * norm.xh).sum(0), g.sum(0)
