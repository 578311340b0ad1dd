"""What surrounds the layer's product, in fp64: activations and their slopes, the
epilogue forward, its backward, and the 8-bit activation checkpoint.

Activation checkpoint (blocks of 64 consecutive values, the last may be
shorter): with c the largest magnitude of a block, d = fl32(c / 127) and
q = fl32(x fl32(127 / c)) rounded to an integer, ties to even; the block stands
for q d.  Blocks with c < 2^-120 are zeros, blocks with an inf or NaN get d = NaN.
"""
import numpy as np
from scipy.special import erfc, expit

CK_BLOCK = 64
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act(z, name):
    """act(z) in fp64."""
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * expit(z)
    if name == "gelu":
        return z * 0.5 * erfc(-z / np.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (z + 0.044715 * z ** 3)))
    raise ValueError(name)


def act_slope(z, name):
    """act'(z) in fp64 (relu'(0) = 0; NaN at NaN)."""
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return np.where(np.isnan(z), z, (z > 0).astype(np.float64))
    if name == "silu":
        p = expit(z)
        return p + z * p * expit(-z)
    if name == "gelu":
        return 0.5 * erfc(-z / np.sqrt(2.0)) + z * np.exp(-z * z / 2.0) / np.sqrt(2.0 * np.pi)
    if name == "gelu_tanh":
        k = np.sqrt(2.0 / np.pi)
        t = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)
    raise ValueError(name)


def ck_quantize(x):
    """Values exactly representable in fp32 (any shape) -> (codes int8 [n], scales float32 [ceil(n / 64)])."""
    x = np.asarray(x, dtype=np.float64).reshape(-1)
    n = x.size
    pad = np.zeros(-(-n // CK_BLOCK) * CK_BLOCK)
    pad[:n] = x
    blk = pad.reshape(-1, CK_BLOCK)
    bad = ~np.isfinite(blk).all(1)
    c = np.abs(np.where(bad[:, None], 0.0, blk)).max(1).astype(np.float32)
    zero = c < np.float32(2.0 ** -120)
    safe = np.where(zero, np.float32(1.0), c)
    d = np.where(zero, np.float32(0.0), c / np.float32(127.0)).astype(np.float32)
    inv = np.where(zero, np.float32(0.0), np.float32(127.0) / safe).astype(np.float32)
    q = np.rint(np.where(bad[:, None], 0.0, blk).astype(np.float32) * inv[:, None])
    d[bad] = np.nan
    return q.astype(np.int8).reshape(-1)[:n], d


def ck_values(codes, scale):
    """fl32(q d) of every code, as fp64."""
    codes = np.asarray(codes, dtype=np.int8)
    d = np.repeat(np.asarray(scale, dtype=np.float32), CK_BLOCK)[:codes.size]
    return (codes.astype(np.float32) * d).astype(np.float64)


def act_fwd(x, w, a, b, scaling, bias=None, name="none", mul=None, residual=None):
    """(Y, Z) in fp64, unrounded; every argument in fp64 (None = absent)."""
    z = x @ w.T
    if a is not None:
        z = z + float(np.float32(scaling)) * ((x @ a) @ b)
    if bias is not None:
        z = z + bias
    y = act(z, name)
    if mul is not None:
        y = y * mul
    if residual is not None:
        y = y + residual
    return y, z


def act_bwd(dy, w, a, b, scaling, name="none", x=None, z=None, mul=None, dx_add=None, round16=None):
    """dict of dx, dmul, dbias, da, db in fp64, unrounded (those that the arguments allow).
    round16: the rounding of dZ to the 16-bit type for the products (dX, dA, dB; the layer's
    definition has it, after dbias); None leaves it out."""
    out, s = {}, float(np.float32(scaling))
    dz = dy
    if mul is not None:
        if z is not None:
            out["dmul"] = dy * act(z, name)
        dz = dz * mul
    if name != "none":
        dz = dz * act_slope(z, name)
    out["dbias"] = dz.sum(0)
    if round16 is not None:
        dz = round16(dz)
    out["dx"] = dz @ w
    if a is not None:
        g = dz @ b.T
        out["dx"] = out["dx"] + s * (g @ a.T)
        if x is not None:
            out["da"] = s * (x.T @ g)
            out["db"] = s * ((x @ a).T @ dz)
    if dx_add is not None:
        out["dx"] = out["dx"] + dx_add
    return out
