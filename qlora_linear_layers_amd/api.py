"""Thin Python binding over the C ABI of ``libqlora_mi355x.so`` (``include/qlora.h``,
``include/qlora_act.h`` and ``include/qlora_block.h``).

Argument marshalling only: every step of the computation runs in the HIP
kernels.  torch provides device memory (tensors) and the current stream.  The
names match the C entry points.  A missing library raises ``RuntimeError``;
there is no fallback.
"""
import ctypes
import math
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora_mi355x.so")

_c_p = ctypes.c_void_p
_c_i64 = ctypes.c_int64
_SIGS = {
    "nf4_build_codebook": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float)]),
    "nf4_quantize_dq": (ctypes.c_int, [_c_p, _c_i64, _c_p, _c_p, _c_p, _c_p]),
    "nf4_dequantize_dq": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_p, _c_p]),
    "qlora_workspace_bytes": (ctypes.c_size_t, [_c_i64, _c_i64, _c_i64, _c_i64]),
    "qlora_workspace_bytes_upto": (ctypes.c_size_t, [_c_i64, _c_i64, _c_i64, _c_i64]),
    "qlora_workspace_bytes_bwd": (ctypes.c_size_t, [_c_i64, _c_i64, _c_i64, _c_i64, ctypes.c_uint]),
    "qlora_linear_fwd": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64,
                                        ctypes.c_float, _c_p, _c_p, ctypes.c_size_t, _c_p]),
    "qlora_linear_bwd_input": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64,
                                              ctypes.c_float, _c_p, _c_p, _c_p, _c_p, _c_p, ctypes.c_size_t,
                                              ctypes.c_uint, _c_p]),
    "qlora_merge_lora": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_i64, ctypes.c_float, _c_p,
                                        _c_p]),
    "nf4_quantize": (ctypes.c_int, [_c_p, _c_i64, _c_p, _c_p, _c_p]),
    "nf4_dequantize": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_p, _c_p]),
    "int4_quantize": (ctypes.c_int, [_c_p, _c_i64, _c_p, _c_p, _c_p]),
    "int4_dequantize": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_p, _c_p]),
    "qlora_linear_fwd_sq": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_i64,
                                           ctypes.c_float, _c_p, _c_p, ctypes.c_size_t, _c_p]),
    "qlora_linear_bwd_input_sq": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_i64,
                                                 ctypes.c_float, _c_p, _c_p, _c_p, _c_p, _c_p, ctypes.c_size_t,
                                                 ctypes.c_uint, _c_p]),
    "qlora_merge_lora_sq": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_i64, ctypes.c_float, _c_p,
                                           _c_p]),
    "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qlora_linear_fwd_noalloc": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64,
                                                ctypes.c_float, _c_p, _c_p]),
    "qlora_noalloc_scratch_bytes": (ctypes.c_size_t, []),
}


class LinearProblem(ctypes.Structure):
    """qlora_linear_problem: one layer of a grouped decode forward."""
    _fields_ = [("x", _c_p), ("codes", _c_p), ("absmax_fp8", _c_p), ("superscale", _c_p), ("lora_a", _c_p),
                ("lora_b", _c_p), ("y", _c_p), ("K", _c_i64), ("N", _c_i64), ("scaling", ctypes.c_float)]


_SIGS["qlora_grouped_workspace_bytes"] = (ctypes.c_size_t, [ctypes.c_int, ctypes.POINTER(LinearProblem), _c_i64,
                                                            _c_i64])
_SIGS["qlora_linear_fwd_grouped"] = (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(LinearProblem), _c_i64, _c_i64,
                                                    _c_p, ctypes.c_size_t, _c_p])
_SIGS["qlora_linear_fwd_grouped_ex"] = (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(LinearProblem), _c_i64, _c_i64,
                                                       ctypes.c_uint, _c_p, ctypes.c_size_t, _c_p])
QLORA_DECODE_MFMA = 1
QLORA_DECODE_VALU = 2


class NF4Tensor(ctypes.Structure):
    """nf4_tensor: one tensor of a grouped quantize / dequantize."""
    _fields_ = [("w", _c_p), ("numel", _c_i64), ("codes", _c_p), ("absmax_fp8", _c_p), ("superscale", _c_p)]


_SIGS["nf4_quantize_dq_grouped"] = (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(NF4Tensor), _c_p])
_SIGS["nf4_dequantize_dq_grouped"] = (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(NF4Tensor), _c_p])
# fp16 compute type: the same arguments as the bf16 entry point of the same stem
for _n in ("nf4_quantize_dq", "nf4_dequantize_dq", "qlora_linear_fwd", "qlora_linear_bwd_input", "qlora_merge_lora"):
    _SIGS[_n + "_f16"] = _SIGS[_n]


class Epilogue(ctypes.Structure):
    """qlora_epilogue: what follows the product in qlora_linear_act_fwd."""
    _fields_ = [("act", ctypes.c_int), ("bias", _c_p), ("mul", _c_p), ("residual", _c_p), ("z", _c_p),
                ("z_codes", _c_p), ("z_scale", _c_p)]


class Saved(ctypes.Structure):
    """qlora_saved: one saved activation, 16-bit values or a checkpoint."""
    _fields_ = [("values", _c_p), ("codes", _c_p), ("scale", _c_p)]


class ActGrad(ctypes.Structure):
    """qlora_act_grad: saved activations and outputs of qlora_linear_act_bwd."""
    _fields_ = [("act", ctypes.c_int), ("x", Saved), ("z", Saved), ("mul", Saved), ("dx_add", _c_p), ("dx", _c_p),
                ("d_lora_a", _c_p), ("d_lora_b", _c_p), ("d_bias", _c_p), ("d_mul", _c_p)]


_SIGS["act8_quantize"] = (ctypes.c_int, [_c_p, _c_i64, _c_p, _c_p, _c_p])
_SIGS["act8_dequantize"] = (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_p, _c_p])
_fwd_tail = [_c_p, _c_p, _c_i64, ctypes.c_float, ctypes.POINTER(Epilogue), _c_p, _c_p, ctypes.c_size_t, _c_p]
_bwd_tail = [_c_p, _c_p, _c_i64, ctypes.c_float, ctypes.POINTER(ActGrad), _c_p, ctypes.c_size_t, _c_p]
for _n, _tail in (("qlora_linear_act_fwd", _fwd_tail), ("qlora_linear_act_bwd", _bwd_tail)):
    _SIGS[_n] = (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p] + _tail)
    _SIGS[_n + "_sq"] = (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p] + _tail)
for _n in ("act8_quantize", "act8_dequantize", "qlora_linear_act_fwd", "qlora_linear_act_bwd"):
    _SIGS[_n + "_f16"] = _SIGS[_n]
_SIGS["qlora_act_workspace_bytes_bwd"] = (ctypes.c_size_t, [_c_i64, _c_i64, _c_i64, _c_i64])
_SIGS["rows8_quantize"] = (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p])
_SIGS["rows8_dequantize"] = (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p])
_SIGS["rmsnorm_fwd"] = (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, ctypes.c_int, ctypes.c_float] + [_c_p] * 5)
_SIGS["rmsnorm_bwd"] = (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, ctypes.c_int, ctypes.c_float] + [_c_p] * 4 +
                        [ctypes.c_size_t, _c_p])
_SIGS["int8_linear_fwd"] = (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, ctypes.POINTER(Epilogue),
                                           _c_p, _c_p, ctypes.c_size_t, _c_p])
for _n in ("rows8_quantize", "rows8_dequantize", "rmsnorm_fwd", "rmsnorm_bwd", "int8_linear_fwd"):
    _SIGS[_n + "_f16"] = _SIGS[_n]
_SIGS["rmsnorm_workspace_bytes_bwd"] = (ctypes.c_size_t, [_c_i64, _c_i64])
_SIGS["int8_linear_workspace_bytes"] = (ctypes.c_size_t, [_c_i64, _c_i64, _c_i64])
EXPORTS = tuple(_SIGS)

REUSE_FORWARD = 1   # QLORA_BWD_REUSE_FORWARD
FUSED_GRADS = 2     # QLORA_BWD_FUSED_GRADS

_lib = None


class QLoraError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed: status {status} ({lib().qlora_status_string(status).decode()})")
        self.status = status


def lib():
    """Load the in-tree HIP library (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(fn, status):
    if status != 0:
        raise QLoraError(fn, status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream():
    """Handle of torch's current stream on the current device (0 is the default stream).  The raw
    getters cost 0.2 us against 2.7 us for torch.cuda.current_stream(), which builds a Stream."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _dev(t, dtype, name):
    if t is None or (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_HALF = (torch.bfloat16, torch.float16)


def _ct(t, name):
    """Compute type of a 16-bit tensor: '' for bf16, '_f16' for fp16."""
    if t.dtype not in _HALF:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return "_f16" if t.dtype == torch.float16 else ""


def _entry(stem, ct, qw):
    """C entry point for a compute type and a storage format."""
    if isinstance(qw, NF4WeightSQ):
        if ct:
            raise ValueError("single quantization has no fp16 entry points")
        return stem + "_sq"
    return stem + ct


def _shape(t, shape, name):
    """Raise ValueError unless tensor `t` (if given) has exactly `shape` (a tuple)."""
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _count(t, n, name):
    """Raise ValueError unless tensor `t` holds exactly `n` elements, in any shape."""
    if t.numel() != n:
        raise ValueError(f"{name} has shape {(t.numel(),)}, expected {(n,)}")


def _check_storage(qw):
    """The storage tensors of a quantized weight must hold exactly what its (N, K) needs:
    the C ABI trusts the sizes, so a mismatch would read past an allocation."""
    n = qw.N * qw.K
    if qw.N < 1 or qw.K < 1 or n % 64:
        raise ValueError(f"quantized weight [{qw.N}, {qw.K}]: N*K must be a positive multiple of 64")
    _count(qw.codes, n // 2, "codes")
    if isinstance(qw, NF4WeightSQ):
        _count(qw.absmax, n // 64, "absmax")
    else:
        _count(qw.absmax_fp8, n // 64, "absmax_fp8")
        _count(qw.superscale, -(-n // 16384), "superscale")


def _dev_storage(qw):
    """The storage of a quantized weight as the kernels read and write it: dense GPU tensors of
    their types (a host address, a narrower type or a strided view of the right count would be
    read past its end)."""
    _dev(qw.codes, torch.uint8, "codes")
    if isinstance(qw, NF4WeightSQ):
        _dev(qw.absmax, torch.float32, "absmax")
    else:
        _dev(qw.absmax_fp8, torch.uint8, "absmax_fp8")
        _dev(qw.superscale, torch.float32, "superscale")


def _dev_workspace(t):
    """A caller's workspace: dense GPU memory of any type, of at least numel() bytes."""
    _dev(t, None if t is None else t.dtype, "workspace")


def _check_adapters(lora_a, lora_b, K, N):
    """Rank of the adapter pair A [K, r], B [r, N] (0 without an adapter)."""
    if (lora_a is None) != (lora_b is None):
        raise ValueError("lora_a and lora_b are given together or not at all")
    if lora_a is None:
        return 0
    if lora_a.dim() != 2:
        raise ValueError(f"lora_a must be 2-D [K, r], got shape {tuple(lora_a.shape)}")
    r = lora_a.shape[1]
    _shape(lora_a, (K, r), "lora_a")
    _shape(lora_b, (r, N), "lora_b")
    return r


@dataclass
class NF4Weight:
    """Storage triple of a quantized [N, K] weight (device tensors)."""
    codes: torch.Tensor       # uint8 [N*K/2]
    absmax_fp8: torch.Tensor  # uint8 [N*K/64]
    superscale: torch.Tensor  # float32 [ceil(N*K/16384)]
    N: int
    K: int

    @property
    def numel(self):
        return self.N * self.K

    def nbytes(self):
        return self.codes.numel() + self.absmax_fp8.numel() + 4 * self.superscale.numel()


@dataclass
class NF4WeightSQ:
    """Single-quantization pair of an [N, K] weight (device tensors): no second level."""
    codes: torch.Tensor       # uint8 [N*K/2]
    absmax: torch.Tensor      # float32 [N*K/64]
    N: int
    K: int

    @property
    def numel(self):
        return self.N * self.K

    def nbytes(self):
        return self.codes.numel() + 4 * self.absmax.numel()


def nf4_build_codebook():
    out = (ctypes.c_float * 16)()
    _check("nf4_build_codebook", lib().nf4_build_codebook(out))
    return torch.tensor(list(out), dtype=torch.float32)


def nf4_quantize_dq(w):
    """bf16 (or fp16) weight [N, K] (or flat) on the GPU -> NF4Weight."""
    ct = _ct(w, "w")
    _dev(w, w.dtype, "w")
    numel = w.numel()
    N, K = (w.shape[0], w.shape[1]) if w.dim() == 2 else (1, numel)
    codes = torch.empty(numel // 2, dtype=torch.uint8, device=w.device)
    fp8 = torch.empty(max(numel // 64, 1), dtype=torch.uint8, device=w.device)
    sup = torch.empty(max(-(-numel // 16384), 1), dtype=torch.float32, device=w.device)
    fn = "nf4_quantize_dq" + ct
    _check(fn, getattr(lib(), fn)(_ptr(w), numel, _ptr(codes), _ptr(fp8), _ptr(sup), _stream()))
    return NF4Weight(codes, fp8, sup, N, K)


def nf4_quantize_dq_into(w, qw):
    """Quantize into an existing NF4Weight (no allocation)."""
    fn = "nf4_quantize_dq" + _ct(w, "w")
    _check_storage(qw)
    if w.numel() != qw.numel:
        raise ValueError(f"w has {w.numel()} elements, the storage holds {qw.numel}")
    _dev(w, w.dtype, "w")
    _dev_storage(qw)
    _check(fn, getattr(lib(), fn)(_ptr(w), w.numel(), _ptr(qw.codes), _ptr(qw.absmax_fp8), _ptr(qw.superscale),
                                  _stream()))


def nf4_dequantize_dq(qw, out=None, dtype=torch.bfloat16):
    """NF4Weight -> [N, K] on the GPU, bf16 or (dtype / out fp16) fp16."""
    _check_storage(qw)
    if out is not None and out.numel() != qw.numel:
        raise ValueError(f"out has {out.numel()} elements, the weight has {qw.numel}")
    if out is None:
        out = torch.empty((qw.N, qw.K), dtype=dtype, device=qw.codes.device)
    fn = "nf4_dequantize_dq" + _ct(out, "out")
    _dev(out, out.dtype, "out")
    _dev_storage(qw)
    _check(fn, getattr(lib(), fn)(_ptr(qw.codes), _ptr(qw.absmax_fp8), _ptr(qw.superscale), qw.numel, _ptr(out),
                                  _stream()))
    return out


MAX_TENSORS = 16         # QLORA_MAX_TENSORS


def _tensor_array(ws, qws):
    if len(ws) != len(qws):
        raise ValueError("one storage triple per weight")
    arr = (NF4Tensor * len(ws))()
    for i, (w, qw) in enumerate(zip(ws, qws)):   # every size first, then the device checks
        _check_storage(qw)
        if w.numel() != qw.numel:
            raise ValueError(f"tensor {i}: {w.numel()} elements, storage for {qw.numel}")
    for i, (w, qw) in enumerate(zip(ws, qws)):
        _dev(w, torch.bfloat16, "w")
        _dev_storage(qw)
        arr[i] = NF4Tensor(w.data_ptr(), w.numel(), qw.codes.data_ptr(), qw.absmax_fp8.data_ptr(),
                           qw.superscale.data_ptr())
    return arr


def nf4_quantize_dq_grouped(ws, qws=None):
    """Quantize up to 16 bf16 weights in one launch; returns (or fills) one NF4Weight per weight."""
    if qws is None:
        qws = []
        for w in ws:
            numel = w.numel()
            N, K = (w.shape[0], w.shape[1]) if w.dim() == 2 else (1, numel)
            qws.append(NF4Weight(torch.empty(numel // 2, dtype=torch.uint8, device=w.device),
                                 torch.empty(max(numel // 64, 1), dtype=torch.uint8, device=w.device),
                                 torch.empty(max(-(-numel // 16384), 1), dtype=torch.float32, device=w.device), N, K))
    _check("nf4_quantize_dq_grouped", lib().nf4_quantize_dq_grouped(len(ws), _tensor_array(ws, qws), _stream()))
    return qws


def nf4_dequantize_dq_grouped(qws, outs=None):
    """Dequantize up to 16 NF4Weights to bf16 in one launch; returns (or fills) the [N, K] outputs."""
    if outs is None:
        outs = [torch.empty((q.N, q.K), dtype=torch.bfloat16, device=q.codes.device) for q in qws]
    _check("nf4_dequantize_dq_grouped", lib().nf4_dequantize_dq_grouped(len(qws), _tensor_array(outs, qws),
                                                                           _stream()))
    return outs


def nf4_quantize(w):
    """bf16 weight [N, K] (or flat) on the GPU -> NF4WeightSQ (single quantization)."""
    _dev(w, torch.bfloat16, "w")
    numel = w.numel()
    N, K = (w.shape[0], w.shape[1]) if w.dim() == 2 else (1, numel)
    codes = torch.empty(numel // 2, dtype=torch.uint8, device=w.device)
    absmax = torch.empty(max(numel // 64, 1), dtype=torch.float32, device=w.device)
    _check("nf4_quantize", lib().nf4_quantize(_ptr(w), numel, _ptr(codes), _ptr(absmax), _stream()))
    return NF4WeightSQ(codes, absmax, N, K)


def nf4_dequantize(qw, out=None):
    """NF4WeightSQ -> bf16 [N, K] on the GPU."""
    _check_storage(qw)
    if out is not None and out.numel() != qw.numel:
        raise ValueError(f"out has {out.numel()} elements, the weight has {qw.numel}")
    if out is None:
        out = torch.empty((qw.N, qw.K), dtype=torch.bfloat16, device=qw.codes.device)
    _dev(out, torch.bfloat16, "out")
    _dev_storage(qw)
    _check("nf4_dequantize", lib().nf4_dequantize(_ptr(qw.codes), _ptr(qw.absmax), qw.numel, _ptr(out), _stream()))
    return out


def int4_quantize(w):
    """bf16 weight on the GPU -> NF4WeightSQ-shaped pair holding INT4 absmax codes (ablation baseline)."""
    _dev(w, torch.bfloat16, "w")
    numel = w.numel()
    N, K = (w.shape[0], w.shape[1]) if w.dim() == 2 else (1, numel)
    codes = torch.empty(numel // 2, dtype=torch.uint8, device=w.device)
    absmax = torch.empty(max(numel // 64, 1), dtype=torch.float32, device=w.device)
    _check("int4_quantize", lib().int4_quantize(_ptr(w), numel, _ptr(codes), _ptr(absmax), _stream()))
    return NF4WeightSQ(codes, absmax, N, K)


def int4_dequantize(qw, out=None):
    _check_storage(qw)
    if out is not None and out.numel() != qw.numel:
        raise ValueError(f"out has {out.numel()} elements, the weight has {qw.numel}")
    if out is None:
        out = torch.empty((qw.N, qw.K), dtype=torch.bfloat16, device=qw.codes.device)
    _dev(out, torch.bfloat16, "out")
    _dev_storage(qw)
    _check("int4_dequantize", lib().int4_dequantize(_ptr(qw.codes), _ptr(qw.absmax), qw.numel, _ptr(out),
                                                     _stream()))
    return out


def _scale_args(qw):
    """(entry-point suffix, block-constant pointers) of either storage format."""
    if isinstance(qw, NF4WeightSQ):
        return "_sq", (_ptr(qw.absmax),)
    return "", (_ptr(qw.absmax_fp8), _ptr(qw.superscale))


def qlora_workspace_bytes(T, K, N, r):
    return int(lib().qlora_workspace_bytes(T, K, N, r))


def qlora_workspace_bytes_upto(T_max, K, N, r):
    """Workspace bytes that serve every call with 1 <= T <= T_max tokens."""
    return int(lib().qlora_workspace_bytes_upto(T_max, K, N, r))


def qlora_workspace_bytes_bwd(T, K, N, r, flags):
    return int(lib().qlora_workspace_bytes_bwd(T, K, N, r, flags))


def workspace_for(T, K, N, r, device):
    n = qlora_workspace_bytes(T, K, N, r)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def qlora_linear_fwd(x, qw, lora_a=None, lora_b=None, scaling=1.0, workspace=None, out=None):
    """Y = X W'^T + scaling (X A) B; x [T, K] -> y [T, N], bf16 or fp16 (the _f16 entry point).
    `qw` is an NF4Weight (double quantization) or an NF4WeightSQ (single quantization, _sq)."""
    ct = _ct(x, "x")
    _check_storage(qw)
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [T, K], got shape {tuple(x.shape)}")
    T, K = x.shape
    _shape(x, (T, qw.K), "x")
    r = _check_adapters(lora_a, lora_b, qw.K, qw.N)
    _shape(out, (T, qw.N), "out")
    _dev(x, x.dtype, "x")
    _dev(lora_a, x.dtype, "lora_a")
    _dev(lora_b, x.dtype, "lora_b")
    _dev_storage(qw)
    _dev_workspace(workspace)
    if out is None:
        out = torch.empty((T, qw.N), dtype=x.dtype, device=x.device)
    if workspace is None:
        workspace = workspace_for(T, K, qw.N, r, x.device)
    _dev(out, x.dtype, "out")
    sc = _scale_args(qw)[1]
    fn = _entry("qlora_linear_fwd", ct, qw)
    _check(fn, getattr(lib(), fn)(
        _ptr(x), T, K, qw.N, _ptr(qw.codes), *sc, _ptr(lora_a), _ptr(lora_b),
        r, float(scaling), _ptr(out), _ptr(workspace), workspace.numel(), _stream()))
    return out


def qlora_linear_fwd_noalloc(x, qw, lora_a=None, lora_b=None, scaling=1.0, out=None):
    """qlora_linear_fwd with the library's static scratch instead of a workspace
    (for callers that cannot allocate; `out` must then be given).  bf16 and
    double quantization only."""
    if x.dtype != torch.bfloat16 or isinstance(qw, NF4WeightSQ):
        raise TypeError("the no-allocation forward takes bf16 tensors and double-quantized weights")
    _check_storage(qw)
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [T, K], got shape {tuple(x.shape)}")
    T = x.shape[0]
    _shape(x, (T, qw.K), "x")
    r = _check_adapters(lora_a, lora_b, qw.K, qw.N)
    _shape(out, (T, qw.N), "out")
    for t, name in ((x, "x"), (lora_a, "lora_a"), (lora_b, "lora_b"), (out, "out")):
        _dev(t, torch.bfloat16, name)
    _dev_storage(qw)
    if out is None:
        out = torch.empty((T, qw.N), dtype=torch.bfloat16, device=x.device)
    _check("qlora_linear_fwd_noalloc", lib().qlora_linear_fwd_noalloc(
        _ptr(x), T, qw.K, qw.N, _ptr(qw.codes), _ptr(qw.absmax_fp8), _ptr(qw.superscale), _ptr(lora_a),
        _ptr(lora_b), r, float(scaling), _ptr(out), _stream()))
    return out


MAX_GROUP = 8            # QLORA_MAX_GROUP
GROUPED_MAX_T = 16       # QLORA_GROUPED_MAX_T


def _grouped_array(problems, T, r):
    arr = (LinearProblem * len(problems))()
    for i, pr in enumerate(problems):          # every shape first, then the device checks
        x, qw, a, b, scaling, y = pr
        if isinstance(qw, NF4WeightSQ):
            raise TypeError("the grouped forward takes double-quantized weights (NF4Weight)")
        _check_storage(qw)
        if tuple(x.shape) != (T, qw.K) or tuple(y.shape) != (T, qw.N):
            raise ValueError(f"problem {i}: x {tuple(x.shape)} / out {tuple(y.shape)} do not match T={T}, "
                             f"K={qw.K}, N={qw.N}")
        if _check_adapters(a, b, qw.K, qw.N) != r:
            raise ValueError(f"problem {i}: every problem of a group has the same rank")
    for i, pr in enumerate(problems):
        x, qw, a, b, scaling, y = pr
        for t, name in ((x, "x"), (a, "lora_a"), (b, "lora_b"), (y, "out")):
            _dev(t, torch.bfloat16, name)
        _dev_storage(qw)
        arr[i] = LinearProblem(x.data_ptr(), qw.codes.data_ptr(), qw.absmax_fp8.data_ptr(), qw.superscale.data_ptr(),
                               None if a is None else a.data_ptr(), None if b is None else b.data_ptr(),
                               y.data_ptr(), qw.K, qw.N, float(scaling))
    return arr


def qlora_grouped_workspace_bytes(problems):
    """Workspace bytes of qlora_linear_fwd_grouped for a list of
    (x, qw, lora_a, lora_b, scaling, out) problems."""
    T = problems[0][0].shape[0]
    r = 0 if problems[0][2] is None else problems[0][2].shape[1]
    arr = _grouped_array(problems, T, r)
    return int(lib().qlora_grouped_workspace_bytes(len(problems), arr, T, r))


def qlora_linear_fwd_grouped(problems, workspace=None, product=None):
    """Decode forward of up to 8 independent layers in one launch pair.  Each
    problem is (x [T, K] bf16, NF4Weight, lora_a or None, lora_b or None,
    scaling, out [T, N] bf16); every problem has the same T (<= 16) and rank.
    Writes each out exactly as qlora_linear_fwd would.  `product` None keeps
    the library's choice; "mfma" or "valu" (T <= 8) picks the decode product
    (qlora_linear_fwd_grouped_ex)."""
    flags = {None: 0, "mfma": QLORA_DECODE_MFMA, "valu": QLORA_DECODE_VALU}.get(product)
    if flags is None:
        raise ValueError(f"product must be None, 'mfma' or 'valu', not {product!r}")
    T = problems[0][0].shape[0]
    r = 0 if problems[0][2] is None else problems[0][2].shape[1]
    arr = _grouped_array(problems, T, r)
    _dev_workspace(workspace)
    if workspace is None:
        n = int(lib().qlora_grouped_workspace_bytes(len(problems), arr, T, r))
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=problems[0][0].device)
    if flags:
        _check("qlora_linear_fwd_grouped_ex", lib().qlora_linear_fwd_grouped_ex(
            len(problems), arr, T, r, flags, _ptr(workspace), workspace.numel(), _stream()))
    else:
        _check("qlora_linear_fwd_grouped", lib().qlora_linear_fwd_grouped(
            len(problems), arr, T, r, _ptr(workspace), workspace.numel(), _stream()))
    return [pr[5] for pr in problems]


def qlora_linear_bwd_input(dy, qw, lora_a=None, lora_b=None, scaling=1.0, x=None, lora_grads=False,
                           workspace=None, dx=None, d_lora_a=None, d_lora_b=None, reuse_forward=False,
                           fused_grads=False):
    """dX (and dA, dB when lora_grads) for upstream gradient dy [T, N] bf16.  With
    reuse_forward, `workspace` must be the one the forward of the same x, A, scaling
    just used (s X A is taken from it).  With fused_grads the dX kernel also forms
    dA and dB (QLORA_BWD_FUSED_GRADS); the workspace must then hold
    qlora_workspace_bytes_bwd(T, K, N, r, flags) bytes."""
    if reuse_forward and workspace is None:
        raise ValueError("reuse_forward needs the forward's workspace")
    ct = _ct(dy, "dy")
    _check_storage(qw)
    if dy.dim() != 2:
        raise ValueError(f"dy must be 2-D [T, N], got shape {tuple(dy.shape)}")
    T, N, K = dy.shape[0], qw.N, qw.K
    _shape(dy, (T, N), "dy")
    r = _check_adapters(lora_a, lora_b, K, N)
    if lora_grads and r == 0:
        raise ValueError("lora_grads needs the adapters")
    if lora_grads and x is None:
        raise ValueError("lora_grads needs x")
    _shape(x, (T, K), "x")
    _shape(dx, (T, K), "dx")
    if lora_grads:
        _shape(d_lora_a, (K, r), "d_lora_a")
        _shape(d_lora_b, (r, N), "d_lora_b")
    _dev(dy, dy.dtype, "dy")
    _dev(x, dy.dtype, "x")
    _dev(lora_a, dy.dtype, "lora_a")
    _dev(lora_b, dy.dtype, "lora_b")
    _dev_storage(qw)
    _dev_workspace(workspace)
    if dx is None:
        dx = torch.empty((T, K), dtype=dy.dtype, device=dy.device)
    if lora_grads:
        if d_lora_a is None:
            d_lora_a = torch.empty((K, r), dtype=dy.dtype, device=dy.device)
        if d_lora_b is None:
            d_lora_b = torch.empty((r, N), dtype=dy.dtype, device=dy.device)
    _dev(dx, dy.dtype, "dx")
    if lora_grads:
        _dev(d_lora_a, dy.dtype, "d_lora_a")
        _dev(d_lora_b, dy.dtype, "d_lora_b")
    flags = (REUSE_FORWARD if reuse_forward else 0) | (FUSED_GRADS if fused_grads else 0)
    if workspace is None:
        n = qlora_workspace_bytes_bwd(T, K, N, r, flags) if fused_grads else qlora_workspace_bytes(T, K, N, r)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=dy.device)
    sc = _scale_args(qw)[1]
    fn = _entry("qlora_linear_bwd_input", ct, qw)
    _check(fn, getattr(lib(), fn)(
        _ptr(dy), T, K, N, _ptr(qw.codes), *sc, _ptr(lora_a), _ptr(lora_b),
        r, float(scaling), _ptr(dx), _ptr(x), _ptr(d_lora_a) if lora_grads else None,
        _ptr(d_lora_b) if lora_grads else None, _ptr(workspace), workspace.numel(), flags, _stream()))
    return (dx, d_lora_a, d_lora_b) if lora_grads else (dx, None, None)


def qlora_merge_lora(qw, lora_a=None, lora_b=None, scaling=1.0, out=None, dtype=None):
    """W_m = RNE_16(W' + scaling (A B)^T) -> [N, K] (W' itself without an adapter), in the
    dtype of the adapters (else of `out`, else `dtype`, else bf16)."""
    dt = lora_a.dtype if lora_a is not None else (out.dtype if out is not None else (dtype or torch.bfloat16))
    _check_storage(qw)
    r = _check_adapters(lora_a, lora_b, qw.K, qw.N)
    _shape(out, (qw.N, qw.K), "out")
    _dev(lora_a, dt, "lora_a")
    _dev(lora_b, dt, "lora_b")
    _dev_storage(qw)
    if out is None:
        out = torch.empty((qw.N, qw.K), dtype=dt, device=qw.codes.device)
    _dev(out, dt, "out")
    sc = _scale_args(qw)[1]
    fn = _entry("qlora_merge_lora", _ct(out, "out"), qw)
    _check(fn, getattr(lib(), fn)(
        _ptr(qw.codes), *sc, qw.K, qw.N, _ptr(lora_a), _ptr(lora_b), r, float(scaling), _ptr(out), _stream()))
    return out


# ------------------------------------------------------------------ epilogue forward, 8-bit checkpoints, their backward

ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}    # QLORA_ACT_*


def _act(name):
    if name not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, not {name!r}")
    return ACTS[name]


class Act8:
    """8-bit checkpoint of an activation (device tensors): `codes` int8 [numel], one per value, and
    `scale` float32 [ceil(numel/64)], one per 64; `shape` is the activation's.  One made by
    act8_empty holds both in a single allocation, and the two tensors are views made when asked for."""
    __slots__ = ("shape", "numel", "_codes", "_scale", "_buf")

    def __init__(self, codes, scale, shape):
        self.shape = tuple(shape)
        self.numel = math.prod(self.shape)
        self._codes, self._scale, self._buf = codes, scale, None

    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._buf[:self.numel]
        return self._codes

    @property
    def scale(self):
        if self._scale is None:
            self._scale = self._buf[-4 * -(-self.numel // 64):].view(torch.float32)
        return self._scale

    @property
    def device(self):
        return (self._codes if self._buf is None else self._buf).device

    def nbytes(self):
        return self.numel + 4 * -(-self.numel // 64)

    def check(self, name):
        """The tensors must hold exactly what the shape needs (an act8_empty's do)."""
        if self._buf is None:
            _count(self._codes, self.numel, name + " codes")
            _count(self._scale, -(-self.numel // 64), name + " scale")

    def pointers(self, name):
        """(codes, scale) addresses of a checkpoint on the GPU."""
        if self._buf is not None:
            if not self._buf.is_cuda:
                raise ValueError(f"{name} codes must be a GPU tensor")
            p = self._buf.data_ptr()
            return p, p + -(-self.numel // 16) * 16
        _dev(self._codes, torch.int8, name + " codes")
        _dev(self._scale, torch.float32, name + " scale")
        return self._codes.data_ptr(), self._scale.data_ptr()


def act8_empty(shape, device="cuda"):
    """An Act8 of uninitialised storage for an activation of `shape`."""
    a8 = Act8(None, None, shape)
    n = a8.numel
    # codes, rounded up to 16 bytes, then the scales
    a8._buf = torch.empty(-(-n // 16) * 16 + 4 * -(-n // 64), dtype=torch.int8, device=device)
    return a8


def act8_quantize(x, out=None):
    """bf16 or fp16 activation of any shape -> Act8 (written into `out` if given)."""
    fn = "act8_quantize" + _ct(x, "x")
    if out is not None:
        out.check("out")
        _shape(x, out.shape, "x")
    _dev(x, x.dtype, "x")
    if out is None:
        out = act8_empty(x.shape, x.device)
    codes, scale = out.pointers("out")
    _check(fn, getattr(lib(), fn)(x.data_ptr(), out.numel, codes, scale, _stream()))
    return out


def act8_dequantize(a8, dtype=torch.bfloat16, out=None):
    """Act8 -> the 16-bit values it stands for, in `dtype` (or in the dtype of `out`)."""
    a8.check("checkpoint")
    _shape(out, a8.shape, "out")
    codes, scale = a8.pointers("checkpoint")
    if out is None:
        out = torch.empty(a8.shape, dtype=dtype, device=a8.device)
    fn = "act8_dequantize" + _ct(out, "out")
    _dev(out, out.dtype, "out")
    _check(fn, getattr(lib(), fn)(codes, scale, a8.numel, out.data_ptr(), _stream()))
    return out


def qlora_linear_act_fwd(x, qw, lora_a=None, lora_b=None, scaling=1.0, bias=None, act="none", mul=None,
                         residual=None, save=None, workspace=None, out=None, z=None):
    """Y = act(Z) * mul + residual with Z = X W'^T + scaling (X A) B + bias; x [T, K] -> y [T, N].
    `act` is one of ACTS; bias [N], mul and residual [T, N] are left out when None.  `out` may be
    the tensor of mul or of residual.  save="z" returns (y, Z) with Z in 16 bits, save="z8" (y,
    Act8 of that Z), for qlora_linear_act_bwd; `z` is the tensor or Act8 to save into."""
    ct = _ct(x, "x")
    code = _act(act)
    if save not in (None, "z", "z8"):
        raise ValueError(f"save must be None, 'z' or 'z8', not {save!r}")
    if z is not None and (save is None or isinstance(z, Act8) != (save == "z8")):
        raise ValueError("z is given with save, a tensor for 'z' and an Act8 for 'z8'")
    _check_storage(qw)
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [T, K], got shape {tuple(x.shape)}")
    T, N, K = x.shape[0], qw.N, qw.K
    _shape(x, (T, K), "x")
    r = _check_adapters(lora_a, lora_b, K, N)
    _shape(bias, (N,), "bias")
    _shape(mul, (T, N), "mul")
    _shape(residual, (T, N), "residual")
    _shape(out, (T, N), "out")
    if z is not None:
        if save == "z8":
            z.check("z")
        if z.shape != (T, N):
            raise ValueError(f"z has shape {tuple(z.shape)}, expected {(T, N)}")
    dt = x.dtype
    _dev(x, dt, "x")
    _dev(lora_a, dt, "lora_a")
    _dev(lora_b, dt, "lora_b")
    _dev(bias, dt, "bias")
    _dev(mul, dt, "mul")
    _dev(residual, dt, "residual")
    _dev(out, dt, "out")
    _dev_storage(qw)
    _dev_workspace(workspace)
    if out is None:
        out = torch.empty((T, N), dtype=dt, device=x.device)
    z16 = zc = zs = None
    if save == "z8":
        if z is None:
            z = act8_empty((T, N), x.device)
        zc, zs = z.pointers("z")
    elif save:
        if z is None:
            z = torch.empty_like(out)
        _dev(z, dt, "z")
        z16 = z.data_ptr()
    if workspace is None:
        workspace = workspace_for(T, K, N, r, x.device)
    ep = Epilogue(code, _ptr(bias), _ptr(mul), _ptr(residual), z16, zc, zs)
    fn = _entry("qlora_linear_act_fwd", ct, qw)
    _check(fn, getattr(lib(), fn)(
        x.data_ptr(), T, K, N, qw.codes.data_ptr(), *_scale_args(qw)[1], _ptr(lora_a), _ptr(lora_b), r,
        float(scaling), ctypes.byref(ep), out.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream()))
    return (out, z) if save else out


@dataclass
class ActGrads:
    """Gradients of qlora_linear_act_bwd; None where not asked for."""
    dx: torch.Tensor
    d_lora_a: torch.Tensor = None
    d_lora_b: torch.Tensor = None
    d_bias: torch.Tensor = None
    d_mul: torch.Tensor = None


def qlora_act_workspace_bytes_bwd(T, K, N, r):
    return int(lib().qlora_act_workspace_bytes_bwd(T, K, N, r))


_ABSENT = Saved()


def _saved(v, shape, name):
    """Checks of one saved activation (tensor, Act8 or None) against its shape."""
    if isinstance(v, Act8):
        v.check(name)
        if v.shape != shape:
            raise ValueError(f"{name} has shape {v.shape}, expected {shape}")
    else:
        _shape(v, shape, name)


def _saved_arg(v, dtype, name):
    """The C argument of a checked saved activation."""
    if v is None:
        return _ABSENT
    if isinstance(v, Act8):
        return Saved(None, *v.pointers(name))
    _dev(v, dtype, name)
    return Saved(v.data_ptr(), None, None)


def _grad_out(t, shape, asked, name):
    """Checks of a caller's gradient tensor, which is given only if it is asked for."""
    if t is not None:
        if not asked:
            raise ValueError(f"{name} is given but its gradient is not asked for")
        _shape(t, shape, name)


def qlora_linear_act_bwd(dy, qw, lora_a=None, lora_b=None, scaling=1.0, act="none", x=None, z=None, mul=None,
                         lora_grads=False, bias_grad=False, mul_grad=True, dx_add=None, workspace=None, dx=None,
                         d_lora_a=None, d_lora_b=None, d_bias=None, d_mul=None):
    """Backward of qlora_linear_act_fwd for upstream gradient dy [T, N] -> ActGrads.  x [T, K], z and
    mul [T, N] are what the forward had (z: before the activation), each a 16-bit tensor or an
    Act8.  x is needed for lora_grads, z for an activation or the gradient of mul (computed when
    mul is given and mul_grad).  dX gets dx_add [T, K] added before its rounding (`dx` may be that
    tensor)."""
    ct = _ct(dy, "dy")
    code = _act(act)
    _check_storage(qw)
    if dy.dim() != 2:
        raise ValueError(f"dy must be 2-D [T, N], got shape {tuple(dy.shape)}")
    T, N, K = dy.shape[0], qw.N, qw.K
    _shape(dy, (T, N), "dy")
    r = _check_adapters(lora_a, lora_b, K, N)
    mul_grad = mul_grad and mul is not None
    if lora_grads and r == 0:
        raise ValueError("lora_grads needs the adapters")
    if lora_grads and x is None:
        raise ValueError("lora_grads needs x")
    if z is None and (code or mul_grad):
        raise ValueError("an activation or the gradient of mul needs z")
    _saved(x, (T, K), "x")
    _saved(z, (T, N), "z")
    _saved(mul, (T, N), "mul")
    _shape(dx_add, (T, K), "dx_add")
    _shape(dx, (T, K), "dx")
    _grad_out(d_lora_a, (K, r), lora_grads, "d_lora_a")
    _grad_out(d_lora_b, (r, N), lora_grads, "d_lora_b")
    _grad_out(d_bias, (N,), bias_grad, "d_bias")
    _grad_out(d_mul, (T, N), mul_grad, "d_mul")
    dt, device = dy.dtype, dy.device
    for t, name in ((dy, "dy"), (lora_a, "lora_a"), (lora_b, "lora_b"), (dx_add, "dx_add"), (dx, "dx"),
                    (d_lora_a, "d_lora_a"), (d_lora_b, "d_lora_b"), (d_bias, "d_bias"), (d_mul, "d_mul")):
        _dev(t, dt, name)
    _dev_storage(qw)
    _dev_workspace(workspace)
    sx, sz, sm = _saved_arg(x, dt, "x"), _saved_arg(z, dt, "z"), _saved_arg(mul, dt, "mul")
    if dx is None:
        dx = torch.empty((T, K), dtype=dt, device=device)
    if lora_grads:
        if d_lora_a is None:
            d_lora_a = torch.empty((K, r), dtype=dt, device=device)
        if d_lora_b is None:
            d_lora_b = torch.empty((r, N), dtype=dt, device=device)
    if bias_grad and d_bias is None:
        d_bias = torch.empty((N,), dtype=dt, device=device)
    if mul_grad and d_mul is None:
        d_mul = torch.empty((T, N), dtype=dt, device=device)
    if workspace is None:
        n = qlora_act_workspace_bytes_bwd(T, K, N, r)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
    g = ActGrad(code, sx, sz, sm, _ptr(dx_add), dx.data_ptr(), _ptr(d_lora_a), _ptr(d_lora_b), _ptr(d_bias),
                _ptr(d_mul))
    fn = _entry("qlora_linear_act_bwd", ct, qw)
    _check(fn, getattr(lib(), fn)(
        dy.data_ptr(), T, K, N, qw.codes.data_ptr(), *_scale_args(qw)[1], _ptr(lora_a), _ptr(lora_b), r,
        float(scaling), ctypes.byref(g), workspace.data_ptr(), workspace.numel(), _stream()))
    return ActGrads(dx, d_lora_a, d_lora_b, d_bias, d_mul)


# ------------------------------------------------------------------ norm, rows in 8 bits, 8-bit integer product

def _on(t, dtype, name, here):
    """A given tensor must be dense, of its type and on the current device `here`, whose stream the
    work goes to."""
    if t is None or (t.dtype is dtype and t.is_contiguous() and t.get_device() == here):
        return
    _dev(t, dtype, name)
    raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{here}")


def _here():
    return torch._C._cuda_getDevice()


def _matrix(t, name):
    """(rows, columns) of a matrix with at least one of each."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(shape)}")
    if shape[0] < 1 or shape[1] < 1:
        raise ValueError(f"{name} has shape {tuple(shape)}: rows and columns must be at least 1")
    return shape


class Rows8:
    """A matrix in 8 bits with one scale per row (device tensors): `codes` int8 [R, P], rows padded by
    zeros to the pitch P (rows8_pitch), and `scale` float32 [R]; `shape` is the matrix's (R, K).  One
    made by rows8_empty holds both in a single allocation, and the two tensors are views made when
    asked for."""
    __slots__ = ("shape", "_codes", "_scale", "_buf")

    def __init__(self, codes, scale, shape):
        self.shape = (int(shape[0]), int(shape[1]))
        self._codes, self._scale, self._buf = codes, scale, None

    @property
    def codes(self):
        if self._codes is None:
            R, P = self.shape[0], rows8_pitch(self.shape[1])
            self._codes = self._buf[:R * P].view(R, P)
        return self._codes

    @property
    def scale(self):
        if self._scale is None:
            self._scale = self._buf[-4 * self.shape[0]:].view(torch.float32)
        return self._scale

    @property
    def device(self):
        return (self._codes if self._buf is None else self._buf).device

    def nbytes(self):
        return self.shape[0] * (rows8_pitch(self.shape[1]) + 4)

    def check(self, name):
        """The tensors must hold exactly what the shape needs (a rows8_empty's do): the C ABI trusts
        the sizes."""
        R, K = self.shape
        if R < 1 or K < 1:
            raise ValueError(f"{name} has shape {self.shape}: rows and columns must be at least 1")
        if self._buf is None:
            _shape(self._codes, (R, rows8_pitch(K)), name + " codes")
            _shape(self._scale, (R,), name + " scale")

    def pointers(self, name, here):
        """(codes, scale) addresses of checked rows on the current device."""
        if self._buf is not None:
            _on(self._buf, torch.int8, name + " codes", here)
            p = self._buf.data_ptr()
            return p, p + self.shape[0] * rows8_pitch(self.shape[1])
        _on(self._codes, torch.int8, name + " codes", here)
        _on(self._scale, torch.float32, name + " scale", here)
        return self._codes.data_ptr(), self._scale.data_ptr()


def rows8_pitch(K):
    """Bytes from one row of codes to the next (QLORA_ROWS8_PITCH)."""
    return -(-K // 128) * 128


def rows8_empty(shape, device="cuda"):
    """A Rows8 of uninitialised storage for a matrix of `shape` (R, K)."""
    r8 = Rows8(None, None, shape)
    R, K = r8.shape
    r8._buf = torch.empty(R * (rows8_pitch(K) + 4), dtype=torch.int8, device=device)     # codes, then scales
    return r8


def rows8_quantize(x, out=None):
    """bf16 or fp16 matrix [R, K] (tokens of an activation, or output channels of a weight) -> Rows8
    (written into `out` if given)."""
    fn = "rows8_quantize" + _ct(x, "x")
    R, K = _matrix(x, "x")
    if out is not None:
        out.check("out")
        _shape(x, out.shape, "x")
    here = _here()
    _on(x, x.dtype, "x", here)
    if out is None:
        out = rows8_empty((R, K), x.device)
    codes, scale = out.pointers("out", here)
    _check(fn, getattr(lib(), fn)(x.data_ptr(), R, K, codes, scale, _stream()))
    return out


def rows8_dequantize(r8, dtype=torch.bfloat16, out=None):
    """Rows8 -> the 16-bit values [R, K] it stands for, in `dtype` (or in the dtype of `out`)."""
    r8.check("rows")
    _shape(out, r8.shape, "out")
    here = _here()
    codes, scale = r8.pointers("rows", here)
    if out is None:
        out = torch.empty(r8.shape, dtype=dtype, device=r8.device)
    else:
        _on(out, out.dtype, "out", here)
    fn = "rows8_dequantize" + _ct(out, "out")
    R, K = r8.shape
    _check(fn, getattr(lib(), fn)(codes, scale, R, K, out.data_ptr(), _stream()))
    return out


def _norm_weight(weight, D, dtype, here):
    """weight_f32 of a norm's weight [D] in the compute type or float32 (or None)."""
    if weight is None:
        return 0
    _shape(weight, (D,), "weight")
    wt = weight.dtype
    if wt is not dtype and wt is not torch.float32:
        raise TypeError(f"weight must be {dtype} or torch.float32, got {wt}")
    _on(weight, wt, "weight", here)
    return int(wt is torch.float32)


def rmsnorm_fwd(x, weight=None, eps=1e-6, residual=None, quantize=False, keep_h=True, h=None, out=None):
    """y = h (mean(h^2) + eps)^(-1/2) weight over the rows of h = x + residual, x [T, D] 16-bit; weight
    [D] in x's dtype or float32, or None for ones.  Returns y, or (y, h) with a residual (`keep_h`
    False drops h); y is a 16-bit tensor or, with `quantize`, the Rows8 of the unrounded y.  `h` and
    `out` are written into if given; `h` may be the tensor of x or of residual."""
    fn = "rmsnorm_fwd" + _ct(x, "x")
    T, D = _matrix(x, "x")
    dt, here = x.dtype, _here()
    if residual is not None:
        _shape(residual, (T, D), "residual")
        _on(residual, dt, "residual", here)
    if h is not None:
        if residual is None or not keep_h:
            raise ValueError("h is given but there is no sum to keep")
        _shape(h, (T, D), "h")
        _on(h, dt, "h", here)
    if out is not None:
        if isinstance(out, Rows8) != bool(quantize):
            raise ValueError("out must be a Rows8 with quantize and a tensor without")
        if quantize:
            out.check("out")
        if tuple(out.shape) != (T, D):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(T, D)}")
    w32 = _norm_weight(weight, D, dt, here)
    _on(x, dt, "x", here)
    if h is None and residual is not None and keep_h:
        h = torch.empty_like(x)
    y = yc = ys = None
    if quantize:
        if out is None:
            out = rows8_empty((T, D), x.device)
        yc, ys = out.pointers("out", here)
    else:
        if out is None:
            out = torch.empty_like(x)
        else:
            _on(out, dt, "out", here)
        y = out.data_ptr()
    _check(fn, getattr(lib(), fn)(x.data_ptr(), _ptr(residual), T, D, _ptr(weight), w32, float(eps), _ptr(h), y, yc, ys,
                                  _stream()))
    return out if h is None else (out, h)


@dataclass
class NormGrads:
    """Gradients of rmsnorm_bwd; d_weight None where not asked for."""
    dx: torch.Tensor
    d_weight: torch.Tensor = None


def rmsnorm_workspace_bytes_bwd(T, D):
    return int(lib().rmsnorm_workspace_bytes_bwd(T, D))


def rmsnorm_bwd(dy, h, weight=None, eps=1e-6, dx_add=None, weight_grad=True, workspace=None, dx=None, d_weight=None):
    """Backward of rmsnorm_fwd for upstream gradient dy [T, D] -> NormGrads.  h is what the forward
    returned (its x without a residual).  dX, the gradient of x and of the residual alike, gets
    dx_add [T, D] (what reaches h on the residual path) added before its rounding; `dx` may be the
    tensor of dy or of dx_add.  d_weight [D] in the weight's dtype, when there is a weight and
    weight_grad."""
    fn = "rmsnorm_bwd" + _ct(dy, "dy")
    T, D = _matrix(dy, "dy")
    dt, here = dy.dtype, _here()
    _shape(h, (T, D), "h")
    weight_grad = weight_grad and weight is not None
    _shape(dx_add, (T, D), "dx_add")
    _shape(dx, (T, D), "dx")
    _grad_out(d_weight, (D,), weight_grad, "d_weight")
    w32 = _norm_weight(weight, D, dt, here)
    _on(dy, dt, "dy", here)
    _on(h, dt, "h", here)
    _on(dx_add, dt, "dx_add", here)
    _on(dx, dt, "dx", here)
    if workspace is not None:
        _on(workspace, workspace.dtype, "workspace", here)
    if dx is None:
        dx = torch.empty_like(dy)
    if weight_grad:
        _on(d_weight, weight.dtype, "d_weight", here)
        if d_weight is None:
            d_weight = torch.empty_like(weight)
        if workspace is None:
            workspace = torch.empty(max(lib().rmsnorm_workspace_bytes_bwd(T, D), 256), dtype=torch.uint8,
                                    device=dy.device)
    _check(fn, getattr(lib(), fn)(dy.data_ptr(), h.data_ptr(), T, D, _ptr(weight), w32, float(eps), _ptr(dx_add),
                                  dx.data_ptr(), _ptr(d_weight), _ptr(workspace),
                                  0 if workspace is None else workspace.numel(), _stream()))
    return NormGrads(dx, d_weight)


def int8_linear_workspace_bytes(T, K, N):
    return int(lib().int8_linear_workspace_bytes(T, K, N))


def int8_linear_fwd(x8, w8, dtype=torch.bfloat16, bias=None, act="none", mul=None, residual=None, workspace=None,
                    out=None):
    """Y = act(X W^T + bias) * mul + residual of two matrices in 8-bit rows: x8 a Rows8 [T, K] (one scale
    per token), w8 a Rows8 [N, K] (one per output channel) -> y [T, N] in `dtype` (or in the dtype
    of `out`).  The product is exact in int32; `act` is one of ACTS; bias [N], mul and residual
    [T, N] in Y's dtype are left out when None.  `out` may be the tensor of mul or of residual."""
    code = _act(act)
    x8.check("x")
    w8.check("w")
    (T, K), N = x8.shape, w8.shape[0]
    if w8.shape[1] != K:
        raise ValueError(f"w has shape {w8.shape}, expected rows of {K}")
    _shape(out, (T, N), "out")
    dt = dtype if out is None else out.dtype
    if dt not in _HALF:
        raise TypeError(f"out must be bfloat16 or float16, got {dt}")
    here = _here()
    for t, shape, name in ((bias, (N,), "bias"), (mul, (T, N), "mul"), (residual, (T, N), "residual")):
        if t is not None:
            _shape(t, shape, name)
            _on(t, dt, name, here)
    xc, xs = x8.pointers("x", here)
    wc, ws = w8.pointers("w", here)
    _on(out, dt, "out", here)
    if out is None:
        like = mul if residual is None else residual
        out = torch.empty((T, N), dtype=dt, device=x8.device) if like is None else torch.empty_like(like)
    L = lib()
    if workspace is None:
        n = L.int8_linear_workspace_bytes(T, K, N)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=x8.device)
    else:
        _on(workspace, workspace.dtype, "workspace", here)
    ep = Epilogue(code, _ptr(bias), _ptr(mul), _ptr(residual), None, None, None)
    fn = "int8_linear_fwd_f16" if dt is torch.float16 else "int8_linear_fwd"
    _check(fn, getattr(L, fn)(
        xc, xs, T, K, N, wc, ws, ctypes.byref(ep), out.data_ptr(), _ptr(workspace),
        0 if workspace is None else workspace.numel(), _stream()))
    return out


# The _sq entry points under their C names (the wrappers above pick them for an NF4WeightSQ).
def qlora_linear_fwd_sq(x, qw, lora_a=None, lora_b=None, scaling=1.0, workspace=None, out=None):
    assert isinstance(qw, NF4WeightSQ)
    return qlora_linear_fwd(x, qw, lora_a, lora_b, scaling, workspace, out)


def qlora_linear_bwd_input_sq(dy, qw, lora_a=None, lora_b=None, scaling=1.0, x=None, lora_grads=False,
                              workspace=None, dx=None, d_lora_a=None, d_lora_b=None, reuse_forward=False,
                              fused_grads=False):
    assert isinstance(qw, NF4WeightSQ)
    return qlora_linear_bwd_input(dy, qw, lora_a, lora_b, scaling, x, lora_grads, workspace, dx, d_lora_a, d_lora_b,
                                  reuse_forward, fused_grads)


def qlora_merge_lora_sq(qw, lora_a=None, lora_b=None, scaling=1.0, out=None):
    assert isinstance(qw, NF4WeightSQ)
    return qlora_merge_lora(qw, lora_a, lora_b, scaling, out)
