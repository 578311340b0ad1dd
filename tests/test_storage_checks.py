"""The binding hands addresses to the C ABI, which cannot tell a host address, a
wider element type or a strided view from what it expects: a quantized weight's
storage and a caller's workspace must be dense GPU tensors of their types before
anything reaches a C entry.  No GPU is needed: the tensors here only say that
they are on one, and the library is a stand-in whose compute entries must not be
reached."""
import pytest
import torch

from qlora_linear_layers_amd import api

N, K, T, R = 1024, 128, 5, 8
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class _OnGpu(torch.Tensor):
    is_cuda = True


class _Library:
    """Sizes are answered, every other entry is a failure."""

    def __getattr__(self, name):
        if "workspace_bytes" in name:
            return lambda *a: 4096

        def entry(*a):
            raise AssertionError(f"reached the C entry {name}")
        return entry


@pytest.fixture(autouse=True)
def _no_library(monkeypatch):
    monkeypatch.setattr(api, "lib", _Library)
    monkeypatch.setattr(api, "_stream", lambda: 0)


def _t(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnGpu)


def _dq(**bad):
    n = N * K
    s = dict(codes=_t(n // 2, dtype=U8), absmax_fp8=_t(n // 64, dtype=U8), superscale=_t(n // 16384, dtype=F32))
    return api.NF4Weight(**{**s, **bad}, N=N, K=K)


def _sq(**bad):
    n = N * K
    s = dict(codes=_t(n // 2, dtype=U8), absmax=_t(n // 64, dtype=F32))
    return api.NF4WeightSQ(**{**s, **bad}, N=N, K=K)


def _calls(qw, workspace=None):
    """Every entry point that reads or writes this weight's storage."""
    x, y, w = _t(T, K), _t(T, N), _t(N, K)
    a, b, ws = _t(K, R), _t(R, N), dict(workspace=workspace)
    calls = {
        "fwd": lambda: api.qlora_linear_fwd(x, qw, a, b, out=y, **ws),
        "bwd": lambda: api.qlora_linear_bwd_input(y, qw, a, b, dx=x, **ws),
        "act_fwd": lambda: api.qlora_linear_act_fwd(x, qw, a, b, out=y, **ws),
        "act_bwd": lambda: api.qlora_linear_act_bwd(y, qw, a, b, dx=x, **ws),
    }
    if isinstance(qw, api.NF4Weight):
        calls["grouped"] = lambda: api.qlora_linear_fwd_grouped([(x, qw, a, b, 0.5, y)], **ws)
    if workspace is not None:
        return calls
    calls["merge"] = lambda: api.qlora_merge_lora(qw, a, b, out=w)
    if isinstance(qw, api.NF4Weight):
        calls["noalloc"] = lambda: api.qlora_linear_fwd_noalloc(x, qw, a, b, out=y)
        calls["dequantize"] = lambda: api.nf4_dequantize_dq(qw, out=w)
        calls["quantize_into"] = lambda: api.nf4_quantize_dq_into(w, qw)
        calls["quantize_grouped"] = lambda: api.nf4_quantize_dq_grouped([w], [qw])
        calls["dequantize_grouped"] = lambda: api.nf4_dequantize_dq_grouped([qw], [w])
    else:
        calls["dequantize"] = lambda: api.nf4_dequantize(qw, out=w)
        calls["int4_dequantize"] = lambda: api.int4_dequantize(qw, out=w)
    return calls


def _plain(t):
    return t.as_subclass(torch.Tensor)


FIELDS = [(_dq, "codes", U8), (_dq, "absmax_fp8", U8), (_dq, "superscale", F32), (_sq, "codes", U8),
          (_sq, "absmax", F32)]


@pytest.mark.parametrize("make,field,dtype", FIELDS)
def test_storage_must_be_dense_gpu_tensors(make, field, dtype):
    n = getattr(make(), field).numel()
    on_host = _plain(getattr(make(), field))
    narrow = _t(n, dtype=torch.int8 if dtype == U8 else torch.float16)
    strided = _t(2 * n, dtype=dtype)[::2]
    for bad, error, match in ((on_host, ValueError, f"{field} must be a GPU tensor"),
                              (narrow, TypeError, f"{field} must be {dtype}"),
                              (strided, ValueError, f"{field} must be contiguous")):
        for name, call in _calls(make(**{field: bad})).items():
            with pytest.raises(error, match=match):
                call()
                pytest.fail(name)


@pytest.mark.parametrize("make", [_dq, _sq])
def test_workspace_must_be_a_dense_gpu_tensor(make):
    for bad, match in ((_plain(_t(1 << 16, dtype=U8)), "workspace must be a GPU tensor"),
                       (_t(1, dtype=U8).expand(1 << 16), "workspace must be contiguous")):
        for name, call in _calls(make(), workspace=bad).items():
            with pytest.raises(ValueError, match=match):
                call()
                pytest.fail(name)


def test_good_storage_reaches_the_library():
    for make in (_dq, _sq):
        for name, call in _calls(make()).items():
            with pytest.raises(AssertionError, match="reached the C entry"):
                call()
