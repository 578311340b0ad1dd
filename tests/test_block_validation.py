"""Refusals of the norm, the 8-bit rows and the 8-bit product: the C entries answer
bad arguments with a status before any launch (fake addresses, never dereferenced),
and the binding checks shapes, options, types and places first (the tensors here
only say that they are on a GPU, and the library behind the binding is a stand-in
whose compute entries must not be reached)."""
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
BF16, F16, F32, I8, U8 = torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.uint8


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(api.LIB_PATH):
        pytest.skip("library not built")
    return api.lib()


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_rows8_refusals(L, suffix):
    for f in (getattr(L, "rows8_quantize" + suffix),
              lambda x, r, k, c, s, st: getattr(L, "rows8_dequantize" + suffix)(c, s, r, k, x, st)):
        assert f(None, 4, 64, FAKE, FAKE, None) == NULL
        assert f(FAKE, 4, 64, None, FAKE, None) == NULL
        assert f(FAKE, 4, 64, FAKE, None, None) == NULL
        for r, k in ((0, 64), (-1, 64), (4, 0), (4, -5), (4, 65537), ((1 << 21) + 1, 64)):
            assert f(FAKE, r, k, FAKE, FAKE, None) == SHAPE, (r, k)
        assert f(MIS, 4, 64, FAKE, FAKE, None) == ALIGN
        assert f(FAKE, 4, 64, MIS, FAKE, None) == ALIGN
        assert f(FAKE, 4, 64, FAKE, MIS, None) == ALIGN


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_norm_refusals(L, suffix):
    def call(x=FAKE, res=FAKE, T=5, D=100, w=FAKE, w32=0, eps=1e-6, h=FAKE, y=FAKE, yc=None, ys=None):
        return getattr(L, "rmsnorm_fwd" + suffix)(x, res, T, D, w, w32, eps, h, y, yc, ys, None)
    assert call(x=None) == NULL and call(y=None) == NULL
    assert call(yc=FAKE) == NULL and call(ys=FAKE) == NULL
    for bad in (dict(T=0), dict(T=-3), dict(T=(1 << 21) + 1), dict(D=0), dict(D=32769)):
        assert call(**bad) == SHAPE, bad
    for k in ("x", "res", "w", "h", "y"):
        assert call(**{k: MIS}) == ALIGN, k
    assert call(yc=MIS, ys=FAKE) == ALIGN and call(yc=FAKE, ys=MIS) == ALIGN
    for eps in (0.0, -1e-6, math.inf, math.nan, 1e-60):       # the last is 0 in fp32
        assert call(eps=eps) == VALUE, eps
    assert call(w32=2) == VALUE and call(w32=1, w=None) == VALUE


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_norm_backward_refusals(L, suffix):
    need = L.rmsnorm_workspace_bytes_bwd(5, 100)
    assert need > 0

    def call(dy=FAKE, h=FAKE, T=5, D=100, w=FAKE, w32=0, eps=1e-6, add=FAKE, dx=FAKE, dw=FAKE, ws=FAKE, wsb=ENOUGH):
        return getattr(L, "rmsnorm_bwd" + suffix)(dy, h, T, D, w, w32, eps, add, dx, dw, ws, wsb, None)
    for k in ("dy", "h", "dx", "w"):
        assert call(**{k: None}) == NULL, k                    # d_weight needs a weight
    for bad in (dict(T=0), dict(D=0), dict(D=32769)):
        assert call(**bad) == SHAPE, bad
        full = {**dict(T=5, D=100), **bad}
        assert L.rmsnorm_workspace_bytes_bwd(full["T"], full["D"]) == 0
    for k in ("dy", "h", "w", "add", "dx", "dw", "ws"):
        assert call(**{k: MIS}) == ALIGN, k
    assert call(eps=0.0) == VALUE and call(w32=-1) == VALUE
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_product_refusals(L, suffix):
    def call(xc=FAKE, xs=FAKE, T=5, K=100, N=70, wc=FAKE, wsc=FAKE, ep=True, y=FAKE, ws=FAKE, wsb=ENOUGH, **e):
        epi = api.Epilogue(**e)
        return getattr(L, "int8_linear_fwd" + suffix)(xc, xs, T, K, N, wc, wsc, ctypes.byref(epi) if ep else None, y, ws,
                                                      wsb, None)
    for k in ("xc", "xs", "wc", "wsc", "y"):
        assert call(**{k: None}) == NULL, k
        assert call(**{k: MIS}) == ALIGN, k
    assert call(ep=False) == NULL and call(ws=MIS) == ALIGN
    for k in ("bias", "mul", "residual"):
        assert call(**{k: MIS}) == ALIGN, k
    for bad in (dict(T=0), dict(K=0), dict(N=0), dict(K=65537), dict(N=(1 << 20) + 1), dict(T=(1 << 21) + 1),
                dict(T=1 << 20, K=2048), dict(T=1 << 20, N=2048)):
        assert call(**bad) == SHAPE, bad
        full = {**dict(T=5, K=100, N=70), **bad}
        assert L.int8_linear_workspace_bytes(full["T"], full["K"], full["N"]) == 0
    assert call(act=-1) == VALUE and call(act=5) == VALUE
    assert call(z=FAKE) == VALUE and call(z_codes=FAKE) == VALUE and call(z_scale=FAKE) == VALUE
    for T, K, N in ((1, 4096, 4096), (300, 4096, 4096), (777, 4096, 128), (64, 65536, 64)):
        need = L.int8_linear_workspace_bytes(T, K, N)
        if need:
            assert call(T=T, K=K, N=N, ws=None) == WORKSPACE and call(T=T, K=K, N=N, wsb=need - 1) == WORKSPACE


# ------------------------------------------------------------------ the binding

class _OnGpu(torch.Tensor):
    is_cuda = True
    device_index = 0

    def get_device(self):
        return self.device_index


class _Library:
    """Sizes are answered, every other entry is a failure."""

    def __getattr__(self, name):
        if "workspace_bytes" in name:
            return lambda *a: 4096

        def entry(*a):
            raise AssertionError(f"reached the C entry {name}")
        return entry


@pytest.fixture
def stub(monkeypatch):
    monkeypatch.setattr(api, "lib", _Library)
    monkeypatch.setattr(api, "_stream", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)


def _t(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnGpu)


def _r8(R, K, codes=None, scale=None):
    return api.Rows8(_t(R, api.rows8_pitch(K), dtype=I8) if codes is None else codes,
                     _t(R, dtype=F32) if scale is None else scale, (R, K))


def _raises(match, fn, *a, **k):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*a, **k)


T, K, N = 5, 100, 70


def test_pitch():
    assert [api.rows8_pitch(k) for k in (1, 127, 128, 129, 4096)] == [128, 128, 128, 256, 4096]


def test_binding_rows8(stub):
    _raises("bfloat16 or float16", api.rows8_quantize, _t(T, K, dtype=F32))
    _raises("2-D", api.rows8_quantize, _t(K))
    for shape in ((0, K), (T, 0)):
        _raises("at least 1", api.rows8_quantize, _t(*shape))
    _raises("x has shape", api.rows8_quantize, _t(T, K), out=_r8(T, K + 1))
    _raises("out codes has shape", api.rows8_quantize, _t(T, K), out=_r8(T, K, codes=_t(T, K, dtype=I8)))
    _raises("out scale has shape", api.rows8_quantize, _t(T, K), out=_r8(T, K, scale=_t(T + 1, dtype=F32)))
    _raises("out codes must be torch.int8", api.rows8_quantize, _t(T, K), out=_r8(T, K, codes=_t(T, 128, dtype=U8)))
    _raises("contiguous", api.rows8_quantize, _t(K, T).t())
    _raises("GPU tensor", api.rows8_quantize, torch.zeros((T, K), dtype=BF16))
    _raises("out has shape", api.rows8_dequantize, _r8(T, K), out=_t(K, T))
    _raises("bfloat16 or float16", api.rows8_dequantize, _r8(T, K), dtype=F32)
    _raises("contiguous", api.rows8_dequantize, _r8(T, K, codes=_t(T, 256, dtype=I8)[:, ::2]), out=_t(T, K))
    _raises("rows scale must be torch.float32", api.rows8_dequantize, _r8(T, K, scale=_t(T, dtype=F16)), out=_t(T, K))


def test_binding_norm(stub):
    f = api.rmsnorm_fwd
    _raises("bfloat16 or float16", f, _t(T, K, dtype=F32))
    _raises("2-D", f, _t(2, T, K))
    _raises("at least 1", f, _t(0, K))
    _raises("weight has shape", f, _t(T, K), _t(T))
    _raises("weight must be torch.bfloat16 or torch.float32", f, _t(T, K), _t(K, dtype=F16))
    _raises("residual has shape", f, _t(T, K), residual=_t(T, K + 1))
    _raises("residual must be torch.bfloat16", f, _t(T, K), residual=_t(T, K, dtype=F16))
    _raises("no sum to keep", f, _t(T, K), h=_t(T, K))
    _raises("no sum to keep", f, _t(T, K), residual=_t(T, K), keep_h=False, h=_t(T, K))
    _raises("h has shape", f, _t(T, K), residual=_t(T, K), h=_t(T + 1, K))
    _raises("out must be a Rows8", f, _t(T, K), quantize=True, out=_t(T, K))
    _raises("out must be a Rows8", f, _t(T, K), out=_r8(T, K))
    _raises("out has shape", f, _t(T, K), quantize=True, out=_r8(T, K + 1))
    _raises("out codes has shape", f, _t(T, K), quantize=True, out=_r8(T, K, codes=_t(T, K, dtype=I8)))
    _raises("out must be torch.bfloat16", f, _t(T, K), out=_t(T, K, dtype=F16))
    _raises("contiguous", f, _t(K, T).t(), out=_t(T, K))
    _raises("GPU tensor", f, _t(T, K), torch.zeros(K, dtype=BF16), out=_t(T, K))
    with pytest.raises(AssertionError, match="reached the C entry rmsnorm_fwd"):
        f(_t(T, K), _t(K, dtype=F32), residual=_t(T, K), h=_t(T, K), out=_t(T, K))


def test_binding_norm_backward(stub):
    f = api.rmsnorm_bwd
    _raises("h has shape", f, _t(T, K), _t(T, K + 1))
    _raises("h must be torch.bfloat16", f, _t(T, K), _t(T, K, dtype=F16))
    _raises("dx_add has shape", f, _t(T, K), _t(T, K), dx_add=_t(K))
    _raises("d_weight is given but", f, _t(T, K), _t(T, K), d_weight=_t(K))
    _raises("d_weight is given but", f, _t(T, K), _t(T, K), _t(K), weight_grad=False, d_weight=_t(K))
    _raises("d_weight must be torch.float32", f, _t(T, K), _t(T, K), _t(K, dtype=F32), d_weight=_t(K))
    _raises("weight must be", f, _t(T, K), _t(T, K), _t(K, dtype=torch.float64))
    _raises("workspace must be contiguous", f, _t(T, K), _t(T, K), _t(K), workspace=_t(1, dtype=U8).expand(1 << 16))
    with pytest.raises(AssertionError, match="reached the C entry rmsnorm_bwd"):
        f(_t(T, K), _t(T, K), dx=_t(T, K))


def test_binding_product(stub):
    f, y = api.int8_linear_fwd, _t(T, N)
    _raises("act must be one of", f, _r8(T, K), _r8(N, K), act="swish")
    _raises("w has shape", f, _r8(T, K), _r8(N, K + 1))
    _raises("x codes has shape", f, _r8(T, K, codes=_t(T, K, dtype=I8)), _r8(N, K))
    _raises("w scale has shape", f, _r8(T, K), _r8(N, K, scale=_t(N, 1, dtype=F32)))
    _raises("x has shape", f, _r8(0, K), _r8(N, K))
    _raises("bias has shape", f, _r8(T, K), _r8(N, K), bias=_t(T))
    _raises("mul has shape", f, _r8(T, K), _r8(N, K), mul=_t(N, T))
    _raises("residual has shape", f, _r8(T, K), _r8(N, K), residual=_t(T, K))
    _raises("out has shape", f, _r8(T, K), _r8(N, K), out=_t(T, K))
    _raises("out must be bfloat16 or float16", f, _r8(T, K), _r8(N, K), dtype=F32)
    _raises("bias must be torch.bfloat16", f, _r8(T, K), _r8(N, K), bias=_t(N, dtype=F16), out=y)
    _raises("w codes must be torch.int8", f, _r8(T, K), _r8(N, K, codes=_t(N, 128, dtype=U8)), out=y)
    _raises("x scale must be a GPU tensor", f, _r8(T, K, scale=torch.zeros(T)), _r8(N, K), out=y)
    _raises("workspace must be a GPU tensor", f, _r8(T, K), _r8(N, K), out=y, workspace=torch.zeros(9, dtype=U8))
    with pytest.raises(AssertionError, match="reached the C entry int8_linear_fwd_f16"):
        f(_r8(T, K), _r8(N, K), mul=_t(T, N, dtype=F16), out=_t(T, N, dtype=F16), workspace=_t(4096, dtype=U8))


def test_binding_refuses_another_device(stub):
    """The work goes to the current device's stream: a tensor elsewhere is refused."""
    def away(t):
        t.device_index = 1
        return t
    w, y = _t(K), _t(T, K)
    for call in (lambda: api.rows8_quantize(away(_t(T, K)), out=_r8(T, K)),
                 lambda: api.rows8_dequantize(_r8(T, K, scale=away(_t(T, dtype=F32))), out=y),
                 lambda: api.rmsnorm_fwd(_t(T, K), away(_t(K)), out=y),
                 lambda: api.rmsnorm_fwd(_t(T, K), w, residual=away(_t(T, K)), h=_t(T, K), out=y),
                 lambda: api.rmsnorm_bwd(_t(T, K), _t(T, K), dx=away(_t(T, K))),
                 lambda: api.int8_linear_fwd(_r8(T, K), _r8(N, K, codes=away(_t(N, 128, dtype=I8))), out=_t(T, N),
                                             workspace=_t(64, dtype=U8))):
        with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
            call()
