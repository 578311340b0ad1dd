"""The root-mean-square norm and its backward, 8-bit rows and the 8-bit product, in fp64.

8-bit rows of a matrix: with c the largest magnitude of a row, d = fl32(c / 127) and
q = fl32(x fl32(127 / c)) rounded to an integer, ties to even; the row stands for q d.  Rows
with c < 2^-120 are zeros, rows with an inf or NaN get d = NaN.  Codes are stored with rows
padded by zeros to a multiple of 128.
"""
import numpy as np

from .act import act

ROWS8_PITCH = 128


def rows8_quantize(x):
    """Values exactly representable in fp32 [R, K] -> (codes int8 [R, pitch], scale float32 [R])."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    bad = ~np.isfinite(x).all(1)
    x = np.where(bad[:, None], 0.0, x).astype(np.float32)
    c = np.abs(x).max(1)
    zero = c < np.float32(2.0 ** -120)
    safe = np.where(zero, np.float32(1.0), c)
    d = np.where(zero, np.float32(0.0), c / np.float32(127.0)).astype(np.float32)
    inv = np.where(zero, np.float32(0.0), np.float32(127.0) / safe).astype(np.float32)
    codes = np.zeros((R, -(-K // ROWS8_PITCH) * ROWS8_PITCH), dtype=np.int8)
    codes[:, :K] = np.rint(x * inv[:, None]).astype(np.int8)
    d[bad] = np.nan
    return codes, d


def rows8_values(codes, scale, K):
    """fl32(q d) of every code, as fp64 [R, K]."""
    codes = np.asarray(codes, dtype=np.int8)[:, :K]
    return (codes.astype(np.float32) * np.asarray(scale, dtype=np.float32)[:, None]).astype(np.float64)


def rmsnorm(h, weight, eps):
    """h (mean(h^2) + eps)^(-1/2) weight over rows; eps as the fp32 it is passed as."""
    h = np.asarray(h, dtype=np.float64)
    r = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + float(np.float32(eps)))
    return h * r if weight is None else h * r * weight


def rmsnorm_bwd(dy, h, weight, eps, dx_add=None):
    """(dx, dw) of rmsnorm's output for upstream dy; dw None without a weight."""
    r = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + float(np.float32(eps)))
    n = h * r
    g = dy if weight is None else dy * weight
    dx = r * (g - n * (g * n).mean(1, keepdims=True))
    if dx_add is not None:
        dx = dx + dx_add
    return dx, None if weight is None else (dy * n).sum(0)


def int8_linear(x_codes, x_scale, w_codes, w_scale, bias=None, name="none", mul=None, residual=None):
    """(Y, Z) in fp64, unrounded, from 8-bit rows (any common pitch); the integer sum is exact."""
    z = x_codes.astype(np.float64) @ w_codes.astype(np.float64).T
    z = z * np.asarray(x_scale, dtype=np.float64)[:, None] * np.asarray(w_scale, dtype=np.float64)[None, :]
    if bias is not None:
        z = z + bias
    y = act(z, name)
    if mul is not None:
        y = y * mul
    if residual is not None:
        y = y + residual
    return y, z
