"""The epilogue forward in every layout of its kernels, each output held to one
rounding.

What a kernel returns is RNE_16(v) with v the fp32 result, so it differs from
RNE_16 of the fp64 reference only where the reference lies within v's error of a
rounding boundary.  That error is at most about 2^-17 of the outputs' rms (the
adapter's intermediates are kept as pairs of 16-bit values in the tiles; fp32
sums and the activations are finer), the boundaries around y are at least u |y|
apart (u the unit roundoff, 2^-8 bf16), and over normal y the mean of
min(1, 2 * 2^-17 rms / (u |y|)) is 2% in bf16: at most 1 value of 33 may differ
there, and no fp16 case (whose pairs are finer too) has more.  An output rounded
once more on its way, for instance an epilogue that starts from a 16-bit Z,
differs in about 2 of 5.  The values that differ are a neighbour: off by no more
than one spacing of the 16-bit type (2 u |y|) plus that error."""
import numpy as np
import pytest
import torch

import oracle
from qlora_linear_layers_amd import api
from helpers import say
from test_gpu_act import U, Case, f64

pytestmark = pytest.mark.gpu


def once(got, ref, what):
    """`got` is RNE_16 of values that agree with `ref` far below their 16-bit spacing."""
    u, r = U[got.dtype], torch.from_numpy(np.ascontiguousarray(ref))
    g, rms = got.double().cpu(), float(r.square().mean().sqrt())
    assert torch.isfinite(g).all(), what
    off = float((g != r.to(got.dtype).double()).double().mean())
    worst = float(((g - r).abs() - 2 * u * r.abs() - 2.0 ** -16 * rms).max())
    say(f"  {what}: {100 * off:.2f}% differ from the rounded reference")
    assert off <= 0.03 and worst <= 0, what


def forward(c, act, bias=True, mul=True, res=True, what=""):
    """Y, Z in both forms, and the in-place forms, of one case."""
    say(f"[epilogue] T={c.T} N={c.N} K={c.K} r={c.r} {act} {what}")
    kw = dict(bias=c.bias if bias else None, act=act, mul=c.mul if mul else None, residual=c.res if res else None)
    y, z = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, save="z", **kw)
    y8, z8 = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, save="z8", **kw)
    q = api.act8_quantize(z)
    plain = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s)
    same = api.qlora_linear_fwd(c.x, c.qw, c.a, c.b, c.s)
    torch.cuda.synchronize()
    ry, rz = oracle.act_fwd(f64(c.x), c.wd, *c.ab64(), c.s, f64(c.bias) if bias else None, act,
                            f64(c.mul) if mul else None, f64(c.res) if res else None)
    once(z, rz, "Z")
    once(y, ry, "Y")
    assert torch.equal(y, y8)
    assert torch.equal(z8.codes, q.codes) and torch.equal(z8.scale, q.scale)
    assert torch.equal(plain.view(torch.int16), same.view(torch.int16))
    for name in [n for n, used in (("mul", mul), ("residual", res)) if used]:
        t = {k: kw[k].clone() for k in ("mul", "residual") if kw[k] is not None}
        out = api.qlora_linear_act_fwd(c.x, c.qw, c.a, c.b, c.s, out=t[name], **{**kw, **t})
        assert out is t[name] and torch.equal(out, y), f"in place of {name}"


# Decode: one column per lane (small launches), two (above 8192 columns, and for more than five
# tokens on a short reduction), one and two tokens per wave, the last 128-column workgroup half
# past N (64 columns past a multiple of 128), several rounds of partials (K above 4096), one and
# several chunks of 64 ranks.
@pytest.mark.parametrize("T,N,K", [(t, n, k) for n, k in ((8256, 192), (320, 4544), (320, 192))
                                   for t in (1, 3, 4, 5, 7, 8, 13)] + [(2, 8256, 4544), (8, 8256, 4544)])
@pytest.mark.parametrize("r,act", [(0, "silu"), (16, "gelu"), (72, "none")])
def test_decode_layouts(T, N, K, r, act):
    forward(Case(T, N, K, r), act)


# Small prefill: two to six 16-token windows, the last one overlapping its predecessor except at
# 48, in one pass over the weight or (few workgroups, at the end) each with its own; the sums'
# launch with two columns per lane (above 16384 columns over the windows) and with one.
@pytest.mark.parametrize("T,N,K", [(17, 8256, 192), (40, 8256, 576), (48, 8256, 192), (63, 8256, 192), (72, 8256, 192),
                                   (96, 8256, 576), (81, 4160, 1088), (72, 1024, 4544), (90, 1024, 4544),
                                   (60, 320, 448), (72, 320, 448), (90, 320, 448)])
@pytest.mark.parametrize("r,act", [(0, "gelu_tanh"), (16, "silu"), (72, "relu")])
def test_window_layouts(T, N, K, r, act):
    forward(Case(T, N, K, r), act)


# Split and whole tiles, ragged in both directions
@pytest.mark.parametrize("T,N,K,r", [(100, 448, 1088, 16), (190, 448, 1088, 0), (300, 448, 1088, 72),
                                     (300, 8256, 192, 16), (520, 4160, 128, 0), (2100, 4160, 64, 8)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_tile_layouts(T, N, K, r, act):
    forward(Case(T, N, K, r), act)


@pytest.mark.parametrize("dtype,storage", [("bf16", "sq"), ("fp16", "dq")])
@pytest.mark.parametrize("T,N,K,r", [(1, 8256, 192, 16), (7, 8256, 576, 8), (7, 320, 192, 8), (7, 320, 4544, 8),
                                     (40, 8256, 192, 16), (72, 8256, 192, 0), (96, 8256, 192, 8), (72, 320, 448, 8),
                                     (300, 448, 1088, 16), (520, 4160, 128, 8)])
def test_types_and_storages(T, N, K, r, dtype, storage):
    forward(Case(T, N, K, r, dtype, storage), "gelu", what=f"{dtype} {storage}")
