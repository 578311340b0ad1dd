"""Refusals of the epilogue forward, the 8-bit checkpoint and the backward from
saved activations: the C entries answer bad arguments with a status before any
launch (fake addresses, never dereferenced), and the Python binding checks every
shape and option first (CPU tensors suffice)."""
import ctypes
import math
import os

import pytest
import torch

from qlora_linear_layers_amd import api

OK, NULL, SHAPE, ALIGN, VALUE, WORKSPACE = 0, 1, 2, 3, 4, 5
FAKE = 1 << 20           # a 16-byte aligned non-NULL address
MIS = FAKE + 8           # misaligned
ENOUGH = 1 << 40
N, K, T, R = 192, 128, 5, 8


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(api.LIB_PATH):
        pytest.skip("library not built")
    return api.lib()


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_checkpoint_refusals(L, suffix):
    for f in (getattr(L, "act8_quantize" + suffix),
              lambda x, n, c, s, st: getattr(L, "act8_dequantize" + suffix)(c, s, n, x, st)):
        assert f(None, 64, FAKE, FAKE, None) == NULL
        assert f(FAKE, 64, None, FAKE, None) == NULL
        assert f(FAKE, 64, FAKE, None, None) == NULL
        for n in (0, -64, (1 << 43) + 1):
            assert f(FAKE, n, FAKE, FAKE, None) == SHAPE
        assert f(MIS, 64, FAKE, FAKE, None) == ALIGN
        assert f(FAKE, 64, MIS, FAKE, None) == ALIGN
        assert f(FAKE, 64, FAKE, MIS, None) == ALIGN


@pytest.mark.parametrize("suffix", ["", "_f16", "_sq"])
def test_forward_refusals(L, suffix):
    scales = [FAKE] if suffix == "_sq" else [FAKE, FAKE]

    def call(T=T, K=K, N=N, r=R, x=FAKE, la=FAKE, lb=FAKE, s=0.5, y=FAKE, ws=FAKE, wsb=ENOUGH, ep=True, **e):
        epi = api.Epilogue(**e)
        return getattr(L, "qlora_linear_act_fwd" + suffix)(
            x, T, K, N, FAKE, *scales, la if r else None, lb if r else None, r, s, ctypes.byref(epi) if ep else None,
            y, ws, wsb, None)
    assert call(ep=False) == NULL
    assert call(x=None) == NULL and call(y=None) == NULL and call(la=None) == NULL
    assert call(z_codes=FAKE) == NULL and call(z_scale=FAKE) == NULL
    for k in ("bias", "mul", "residual", "z"):
        assert call(**{k: MIS}) == ALIGN, k
    assert call(z_codes=MIS, z_scale=FAKE) == ALIGN and call(z_codes=FAKE, z_scale=MIS) == ALIGN
    assert call(act=-1) == VALUE and call(act=5) == VALUE
    assert call(s=math.nan) == VALUE and call(s=math.inf) == VALUE
    for bad in (dict(T=0), dict(T=-1), dict(K=100), dict(N=32), dict(r=12), dict(r=264), dict(T=1 << 23),
                dict(T=1 << 20, K=2048)):
        assert call(**bad) == SHAPE, bad
    assert call(ws=None) == WORKSPACE and call(wsb=16) == WORKSPACE
    assert call(T=300, ws=None) == WORKSPACE and call(ws=MIS) == ALIGN


@pytest.mark.parametrize("suffix", ["", "_f16", "_sq"])
def test_backward_refusals(L, suffix):
    scales = [FAKE] if suffix == "_sq" else [FAKE, FAKE]
    assert L.qlora_act_workspace_bytes_bwd(T, K, N, R) > 0
    # 300 tokens: the backward's own need is larger than the forward's there
    need300 = L.qlora_act_workspace_bytes_bwd(300, K, N, R)
    v16, ck = api.Saved(FAKE, None, None), api.Saved(None, FAKE, FAKE)

    def call(T=T, K=K, N=N, r=R, dy=FAKE, la=FAKE, lb=FAKE, s=0.5, ws=FAKE, wsb=ENOUGH, grad=True, dx=FAKE, **g):
        a = api.ActGrad(dx=dx, **g)
        return getattr(L, "qlora_linear_act_bwd" + suffix)(
            dy, T, K, N, FAKE, *scales, la if r else None, lb if r else None, r, s, ctypes.byref(a) if grad else None,
            ws, wsb, None)
    assert call(grad=False) == NULL and call(dy=None) == NULL and call(dx=None) == NULL and call(lb=None) == NULL
    # a required activation missing
    assert call(d_lora_a=FAKE) == NULL and call(d_lora_b=FAKE) == NULL
    assert call(act=2) == NULL and call(d_mul=FAKE, z=ck) == NULL and call(d_mul=FAKE, mul=ck) == NULL
    # half a checkpoint, both forms at once
    for k in ("x", "z", "mul"):
        assert call(**{k: api.Saved(None, FAKE, None)}) == NULL, k
        assert call(**{k: api.Saved(None, None, FAKE)}) == NULL, k
        assert call(**{k: api.Saved(FAKE, FAKE, FAKE)}) == VALUE, k
        assert call(**{k: api.Saved(MIS, None, None)}) == ALIGN, k
        assert call(**{k: api.Saved(None, MIS, FAKE)}) == ALIGN, k
    for k in ("dx_add", "dx", "d_bias"):
        assert call(**{k: MIS}) == ALIGN, k
    assert call(d_lora_a=MIS, x=v16) == ALIGN and call(d_mul=MIS, z=ck, mul=ck) == ALIGN
    assert call(r=0, d_lora_a=FAKE, x=v16) == SHAPE
    for bad in (dict(T=0), dict(K=100), dict(N=32), dict(r=12), dict(T=1 << 23)):
        assert call(**bad) == SHAPE, bad
        full = {**dict(T=T, K=K, N=N, r=R), **bad}
        assert L.qlora_act_workspace_bytes_bwd(full["T"], full["K"], full["N"], full["r"]) == 0
    assert call(act=5, z=ck) == VALUE and call(act=-1, z=ck) == VALUE and call(s=math.inf) == VALUE
    assert call(ws=None) == WORKSPACE and call(T=300, wsb=need300 - 1) == WORKSPACE


def test_backward_workspace_covers_the_plain_backward(L):
    for t in (1, 16, 17, 96, 97, 300, 2048, 9001):
        for k, n, r in ((64, 64, 0), (4096, 11008, 64), (11008, 4096, 24)):
            assert L.qlora_act_workspace_bytes_bwd(t, k, n, r) >= L.qlora_workspace_bytes_bwd(t, k, n, r, 0)


# ------------------------------------------------------------------ the binding

def _qw():
    n = N * K
    return api.NF4Weight(torch.zeros(n // 2, dtype=torch.uint8), torch.zeros(n // 64, dtype=torch.uint8),
                         torch.zeros(-(-n // 16384), dtype=torch.float32), N, K)


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _a8(*shape, short=0):
    n = math.prod(shape)
    return api.Act8(_t(n - short, dtype=torch.int8), _t(-(-n // 64), dtype=torch.float32), shape)


def _raises(fn, match):
    with pytest.raises((ValueError, TypeError), match=match):
        fn()


def test_binding_forward_refusals():
    qw, x = _qw(), _t(T, K)
    f = lambda *a, **k: lambda: api.qlora_linear_act_fwd(*a, **k)
    _raises(f(x, qw, act="swish"), "act must be one of")
    _raises(f(x, qw, save="z16"), "save must be")
    _raises(f(x, qw, z=_t(T, N)), "z is given with save")
    _raises(f(x, qw, save="z", z=_a8(T, N)), "z is given with save")
    _raises(f(x, qw, save="z8", z=_a8(T, N, short=1)), "z codes has shape")
    _raises(f(x, qw, save="z8", z=_a8(T, N + 64)), "z has shape")
    _raises(f(_t(T, K + 64), qw), "x has shape")
    _raises(f(x, qw, bias=_t(N + 64)), "bias has shape")
    _raises(f(x, qw, mul=_t(T + 1, N)), "mul has shape")
    _raises(f(x, qw, residual=_t(T, K)), "residual has shape")
    _raises(f(x, qw, out=_t(T, K)), "out has shape")
    _raises(f(x, qw), "GPU tensor")
    _raises(f(x.float(), qw), "bfloat16 or float16")


def test_binding_backward_refusals():
    qw, dy = _qw(), _t(T, N)
    a, b = _t(K, R), _t(R, N)
    f = lambda *p, **k: lambda: api.qlora_linear_act_bwd(*p, **k)
    _raises(f(_t(T, K), qw), "dy has shape")
    _raises(f(dy, qw, act="silu"), "needs z")
    _raises(f(dy, qw, mul=_a8(T, N)), "needs z")
    _raises(f(dy, qw, lora_grads=True), "needs the adapters")
    _raises(f(dy, qw, a, b, lora_grads=True), "needs x")
    _raises(f(dy, qw, a, b, x=_a8(T, N), lora_grads=True), "x has shape")
    _raises(f(dy, qw, act="silu", z=_a8(T, K)), "z has shape")
    _raises(f(dy, qw, act="silu", z=_a8(T, N), mul=_t(T, K)), "mul has shape")
    _raises(f(dy, qw, act="silu", z=_a8(T, N, short=2)), "z codes has shape")
    _raises(f(dy, qw, dx_add=_t(T, N)), "dx_add has shape")
    _raises(f(dy, qw, d_bias=_t(N)), "not asked for")
    _raises(f(dy, qw, bias_grad=True, d_bias=_t(K)), "d_bias has shape")
    _raises(f(dy, qw), "GPU tensor")


def test_binding_checkpoint_refusals():
    _raises(lambda: api.act8_quantize(_t(3, dtype=torch.float32)), "bfloat16 or float16")
    _raises(lambda: api.act8_quantize(_t(3, 5)), "GPU tensor")
    _raises(lambda: api.act8_quantize(_t(3, 5), out=_a8(3, 6)), "x has shape")
    _raises(lambda: api.act8_quantize(_t(3, 5), out=_a8(3, 5, short=1)), "out codes has shape")
    _raises(lambda: api.act8_dequantize(_a8(3, 5, short=1)), "checkpoint codes has shape")
    _raises(lambda: api.act8_dequantize(_a8(3, 5), out=_t(5, 3)), "out has shape")
    _raises(lambda: api.act8_dequantize(_a8(3, 5)), "GPU tensor")
