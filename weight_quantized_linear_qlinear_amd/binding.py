"""ctypes binding of libqlq.so: argument marshalling only.

Every function here checks shapes and dtypes, allocates outputs with PyTorch on
the tensors' device, and forwards plain pointers, sizes and the current HIP
stream to the C ABI declared in include/qlq.h.  All arithmetic runs in the HIP
kernels; there is no fallback path: if the library is not built, or the tensors
are not on a GPU, the call raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import math
import os
import threading

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqlq.so")

QTYPES = {"int8": 0, "fp8_e4m3fn": 1}
GRANULARITIES = {"per_channel": 0, "per_tensor": 1}
OUTS = {"bf16": 0, "acc": 1}
SCHEMES = {"w8a16": 0, "w8a8_static": 1, "w8a8_static_fused": 2, "w8a8_dynamic": 3}
STATUS = {0: "QLQ_OK", 1: "QLQ_ERR_INVALID_ARG", 2: "QLQ_ERR_UNSUPPORTED", 3: "QLQ_ERR_HIP"}

# name -> (restype, argtypes), mirroring include/qlq.h
_c = ctypes
_SIGNATURES = {
    "qlq_packed_weight_bytes": (_c.c_size_t, [_c.c_int64, _c.c_int64]),
    "qlq_workspace_bytes": (_c.c_size_t, [_c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int]),
    "qlq_quantize_weight": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int,
                                       _c.c_void_p, _c.c_void_p, _c.c_void_p]),
    "qlq_unpack_weight": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_void_p]),
    "qlq_calibrate_input_scale": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_int, _c.c_void_p, _c.c_void_p]),
    "qlq_quantize_act_static": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_float, _c.c_int,
                                           _c.c_void_p, _c.c_void_p]),
    "qlq_qlinear_w8a16": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_void_p,
                                     _c.c_int64, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "qlq_qlinear_w8a16_noalloc": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p,
                                             _c.c_void_p, _c.c_int64, _c.c_int, _c.c_void_p, _c.c_void_p]),
    "qlq_qlinear_w8a8_static": (_c.c_int, [_c.c_void_p, _c.c_float, _c.c_int64, _c.c_int64, _c.c_int64,
                                           _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int, _c.c_int,
                                           _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "qlq_qlinear_w8a8_static_requant": (_c.c_int, [_c.c_void_p, _c.c_float, _c.c_int64, _c.c_int64, _c.c_int64,
                                                   _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int, _c.c_float,
                                                   _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t,
                                                   _c.c_void_p]),
    "qlq_quantize_act_dynamic": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int, _c.c_void_p,
                                            _c.c_void_p, _c.c_void_p]),
    "qlq_qlinear_w8a8_static_fused": (_c.c_int, [_c.c_void_p, _c.c_float, _c.c_int64, _c.c_int64, _c.c_int64,
                                                 _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int, _c.c_int,
                                                 _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "qlq_qlinear_w8a8_dynamic": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64,
                                            _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int, _c.c_int,
                                            _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "qlq_kv_quantize": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p,
                                   _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p]),
    "qlq_kv_dequantize": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64,
                                     _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_void_p]),
    "qlq_rms_norm": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_float,
                                _c.c_void_p, _c.c_void_p, _c.c_void_p]),
    "qlq_rms_norm_quant_static": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64,
                                             _c.c_float, _c.c_float, _c.c_int, _c.c_void_p, _c.c_void_p,
                                             _c.c_void_p]),
    "qlq_rms_norm_quant_dynamic": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64,
                                              _c.c_float, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                              _c.c_void_p]),
    "qlq_rope": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int,
                            _c.c_void_p, _c.c_int64, _c.c_float, _c.c_int, _c.c_void_p, _c.c_int64, _c.c_void_p]),
    "qlq_kv_append": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64,
                                 _c.c_int64, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_void_p, _c.c_void_p,
                                 _c.c_void_p, _c.c_void_p, _c.c_void_p]),
    "qlq_rope_kv_append": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64,
                                      _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int,
                                      _c.c_void_p, _c.c_int64, _c.c_float, _c.c_int, _c.c_void_p, _c.c_int,
                                      _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                      _c.c_int64, _c.c_void_p]),
    "qlq_kv_gather": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int64,
                                 _c.c_int64, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_void_p, _c.c_void_p,
                                 _c.c_void_p]),
    "qlq_kv_attention": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64,
                                    _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64,
                                    _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_float,
                                    _c.c_int, _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t,
                                    _c.c_void_p]),
    "qlq_kv_attention_workspace_bytes": (_c.c_size_t, [_c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64,
                                                       _c.c_int]),
    "qlq_linear": (_c.c_int, [_c.c_int, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_void_p,
                              _c.c_int64, _c.c_int, _c.c_float, _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_void_p,
                              _c.c_size_t, _c.c_void_p]),
    "qlq_linear_workspace_bytes": (_c.c_size_t, [_c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int]),
    "qlq_gemm_plan": (_c.c_int, [_c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int, _c.c_void_p]),
    "qlq_scale_is_calibrated": (_c.c_int, [_c.c_float]),
    "qlq_status_string": (_c.c_char_p, [_c.c_int]),
    "qlq_last_error": (_c.c_char_p, []),
    "qlq_version": (_c.c_char_p, []),
}

_lib = None
_lock = threading.Lock()


class QlqError(RuntimeError):
    """A non-OK status from libqlq (validation or launch failure)."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libqlq.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(_LIB_PATH):
                    raise ImportError(f"{_LIB_PATH} is missing: build it with "
                                      "`python -m weight_quantized_linear_qlinear_amd.build`")
                h = ctypes.CDLL(_LIB_PATH)
                for name, (res, args) in _SIGNATURES.items():
                    f = getattr(h, name)
                    f.restype = res
                    f.argtypes = args
                _lib = h
    return _lib


def _check(status: int):
    if status != 0:
        raise QlqError(status, lib().qlq_last_error().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _require_gpu(*ts: torch.Tensor):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("qlq operates on GPU tensors only")
        if not t.is_contiguous():
            raise ValueError("qlq needs contiguous (row-major) tensors")


def _qtype(q: str) -> int:
    if q not in QTYPES:
        raise ValueError(f"qtype must be one of {sorted(QTYPES)}")
    return QTYPES[q]


def code_dtype(qtype: str) -> torch.dtype:
    """torch dtype used for 1-byte codes: int8 for INT8, uint8 (raw bits) for e4m3fn."""
    return torch.int8 if qtype == "int8" else torch.uint8


# ---------------------------------------------------------------------- sizing
def packed_weight_bytes(N: int, K: int) -> int:
    return int(lib().qlq_packed_weight_bytes(N, K))


def workspace_bytes(scheme: str, M: int, K: int, N: int, qtype: str) -> int:
    return int(lib().qlq_workspace_bytes(SCHEMES[scheme], M, K, N, _qtype(qtype)))


class _PlanInfo(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("cfg", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("waves", ctypes.c_int32),
                ("grid", ctypes.c_int32), ("workspace_bytes", ctypes.c_int64)]


def gemm_plan(scheme: str, M: int, K: int, N: int, qtype: str) -> dict:
    """The launch plan a GEMM call takes for these sizes (test hook; host only)."""
    info = _PlanInfo()
    _check(lib().qlq_gemm_plan(SCHEMES[scheme], M, K, N, _qtype(qtype), ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in _PlanInfo._fields_}


def scale_is_calibrated(s: float) -> bool:
    """Whether the quantizers take the refined-reciprocal division for scale s (test hook)."""
    return bool(lib().qlq_scale_is_calibrated(float(s)))


_workspaces: dict = {}


def _workspace(dev: torch.device, nbytes: int) -> torch.Tensor | None:
    """A zero-filled per-device workspace, grown on demand (the kernels leave it zeroed)."""
    if nbytes == 0:
        return None
    key = (dev.type, dev.index)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws


# ---------------------------------------------------------------------- weights
@dataclasses.dataclass
class QuantizedWeight:
    """A packed quantized weight of logical shape [N, K] and its fp32 scales."""
    packed: torch.Tensor      # uint8, packed_weight_bytes(N, K)
    scale: torch.Tensor       # fp32 [N] (per channel) or [1] (per tensor)
    N: int
    K: int
    qtype: str
    granularity: str


def quantize_weight(w: torch.Tensor, qtype: str, granularity: str = "per_channel",
                    packed: torch.Tensor | None = None, scale: torch.Tensor | None = None) -> QuantizedWeight:
    """Quantize and pack W[N, K] (fp32 or bf16, on the GPU)."""
    _require_gpu(w)
    if w.dim() != 2 or w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("w must be a 2-D fp32 or bf16 tensor")
    N, K = w.shape
    if granularity not in GRANULARITIES:
        raise ValueError(f"granularity must be one of {sorted(GRANULARITIES)}")
    if packed is None:
        packed = torch.empty(packed_weight_bytes(N, K), dtype=torch.uint8, device=w.device)
    if scale is None:
        scale = torch.empty(N if granularity == "per_channel" else 1, dtype=torch.float32, device=w.device)
    _check(lib().qlq_quantize_weight(_ptr(w), int(w.dtype == torch.bfloat16), N, K, _qtype(qtype),
                                     GRANULARITIES[granularity], _ptr(packed), _ptr(scale), _stream(w.device)))
    return QuantizedWeight(packed, scale, N, K, qtype, granularity)


def unpack_weight(qw: QuantizedWeight) -> torch.Tensor:
    """Row-major [N, K] codes of a packed weight (test hook)."""
    out = torch.empty((qw.N, qw.K), dtype=code_dtype(qw.qtype), device=qw.packed.device)
    _check(lib().qlq_unpack_weight(_ptr(qw.packed), qw.N, qw.K, _ptr(out), _stream(out.device)))
    return out


# ---------------------------------------------------------------------- activations
def calibrate_input_scale(x_calib: torch.Tensor, qtype: str, out: torch.Tensor | None = None) -> torch.Tensor:
    """Static input scale absmax(x_calib) / qmax as a one-element fp32 device tensor."""
    _require_gpu(x_calib)
    if x_calib.dtype != torch.bfloat16:
        raise ValueError("x_calib must be bf16")
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x_calib.device)
    _check(lib().qlq_calibrate_input_scale(_ptr(x_calib), x_calib.numel(), _qtype(qtype), _ptr(out),
                                           _stream(x_calib.device)))
    return out


def quantize_act_static(x: torch.Tensor, input_scale: float, qtype: str,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """Codes of x [M, K] bf16 with the fixed scalar input_scale."""
    _require_gpu(x)
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise ValueError("x must be a 2-D bf16 tensor")
    M, K = x.shape
    if out is None:
        out = torch.empty((M, K), dtype=code_dtype(qtype), device=x.device)
    _check(lib().qlq_quantize_act_static(_ptr(x), M, K, float(input_scale), _qtype(qtype), _ptr(out),
                                         _stream(x.device)))
    return out


def quantize_act_dynamic(x: torch.Tensor, qtype: str, out: torch.Tensor | None = None,
                         x_scale: torch.Tensor | None = None):
    """Per-token codes of x [M, K] bf16 and their row scales: (xq [M, K], x_scale fp32 [M])."""
    _require_gpu(x)
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise ValueError("x must be a 2-D bf16 tensor")
    M, K = x.shape
    if out is None:
        out = torch.empty((M, K), dtype=code_dtype(qtype), device=x.device)
    if x_scale is None:
        x_scale = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib().qlq_quantize_act_dynamic(_ptr(x), M, K, _qtype(qtype), _ptr(out), _ptr(x_scale),
                                          _stream(x.device)))
    return out, x_scale


# ---------------------------------------------------------------------- GEMMs
def qlinear_w8a16(x: torch.Tensor, qw: QuantizedWeight, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = x W^T with W dequantized to bf16 in the kernel; x bf16 [M, K] -> y bf16 [M, N]."""
    _require_gpu(x)
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.shape[1] != qw.K:
        raise ValueError(f"x must be bf16 [M, {qw.K}]")
    M = x.shape[0]
    if out is None:
        out = torch.empty((M, qw.N), dtype=torch.bfloat16, device=x.device)
    nbytes = workspace_bytes("w8a16", M, qw.K, qw.N, qw.qtype)
    ws = workspace if workspace is not None else _workspace(x.device, nbytes)
    _check(lib().qlq_qlinear_w8a16(_ptr(x), M, qw.K, qw.N, _ptr(qw.packed), _ptr(qw.scale), qw.scale.numel(),
                                   _qtype(qw.qtype), _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(),
                                   _stream(x.device)))
    return out


def qlinear_w8a16_noalloc(x: torch.Tensor, qw: QuantizedWeight, out: torch.Tensor) -> torch.Tensor:
    """qlinear_w8a16 without a workspace (split-K scratch inside the library); out is required."""
    _require_gpu(x, out)
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.shape[1] != qw.K:
        raise ValueError(f"x must be bf16 [M, {qw.K}]")
    M = x.shape[0]
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (M, qw.N):
        raise ValueError(f"out must be bf16 [{M}, {qw.N}]")
    _check(lib().qlq_qlinear_w8a16_noalloc(_ptr(x), M, qw.K, qw.N, _ptr(qw.packed), _ptr(qw.scale),
                                           qw.scale.numel(), _qtype(qw.qtype), _ptr(out), _stream(x.device)))
    return out


def qlinear_w8a8_static(xq: torch.Tensor, input_scale: float, qw: QuantizedWeight, out_mode: str = "bf16",
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """W8A8 static GEMM on codes xq [M, K]: bf16 y [M, N], or raw accumulators (out_mode="acc")."""
    _require_gpu(xq)
    if xq.dim() != 2 or xq.element_size() != 1 or xq.shape[1] != qw.K:
        raise ValueError(f"xq must be 1-byte codes [M, {qw.K}]")
    M = xq.shape[0]
    if out is None:
        if out_mode == "acc":
            dt = torch.int32 if qw.qtype == "int8" else torch.float32
        else:
            dt = torch.bfloat16
        out = torch.empty((M, qw.N), dtype=dt, device=xq.device)
    nbytes = workspace_bytes("w8a8_static", M, qw.K, qw.N, qw.qtype)
    ws = workspace if workspace is not None else _workspace(xq.device, nbytes)
    _check(lib().qlq_qlinear_w8a8_static(_ptr(xq), float(input_scale), M, qw.K, qw.N, _ptr(qw.packed),
                                         _ptr(qw.scale), qw.scale.numel(), _qtype(qw.qtype), OUTS[out_mode],
                                         _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(),
                                         _stream(xq.device)))
    return out


def qlinear_w8a8_static_requant(xq: torch.Tensor, input_scale: float, qw: QuantizedWeight, next_scale: float,
                                out: torch.Tensor | None = None, out_codes: torch.Tensor | None = None,
                                workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """W8A8 static GEMM on codes xq [M, K] that also quantizes its bf16 output for the next static layer:
    returns (y bf16 [M, N], codes [M, N] of y at next_scale, same qtype)."""
    _require_gpu(xq)
    if xq.dim() != 2 or xq.element_size() != 1 or xq.shape[1] != qw.K:
        raise ValueError(f"xq must be 1-byte codes [M, {qw.K}]")
    M = xq.shape[0]
    if out is None:
        out = torch.empty((M, qw.N), dtype=torch.bfloat16, device=xq.device)
    if out_codes is None:
        out_codes = torch.empty((M, qw.N), dtype=code_dtype(qw.qtype), device=xq.device)
    if out_codes.shape != (M, qw.N) or out_codes.element_size() != 1:
        raise ValueError(f"out_codes must be 1-byte codes [{M}, {qw.N}]")
    nbytes = workspace_bytes("w8a8_static", M, qw.K, qw.N, qw.qtype)
    ws = workspace if workspace is not None else _workspace(xq.device, nbytes)
    _check(lib().qlq_qlinear_w8a8_static_requant(_ptr(xq), float(input_scale), M, qw.K, qw.N, _ptr(qw.packed),
                                                 _ptr(qw.scale), qw.scale.numel(), _qtype(qw.qtype),
                                                 float(next_scale), _ptr(out), _ptr(out_codes), _ptr(ws),
                                                 0 if ws is None else ws.numel(), _stream(xq.device)))
    return out, out_codes


def _w8a8_out(M: int, qw: QuantizedWeight, out_mode: str, dev: torch.device) -> torch.Tensor:
    if out_mode == "acc":
        dt = torch.int32 if qw.qtype == "int8" else torch.float32
    else:
        dt = torch.bfloat16
    return torch.empty((M, qw.N), dtype=dt, device=dev)


def qlinear_w8a8_static_fused(x: torch.Tensor, input_scale: float, qw: QuantizedWeight, out_mode: str = "bf16",
                              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """quantize_act_static + qlinear_w8a8_static in one call, from bf16 x [M, K]."""
    _require_gpu(x)
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.shape[1] != qw.K:
        raise ValueError(f"x must be bf16 [M, {qw.K}]")
    M = x.shape[0]
    if out is None:
        out = _w8a8_out(M, qw, out_mode, x.device)
    nbytes = workspace_bytes("w8a8_static_fused", M, qw.K, qw.N, qw.qtype)
    ws = workspace if workspace is not None else _workspace(x.device, nbytes)
    _check(lib().qlq_qlinear_w8a8_static_fused(_ptr(x), float(input_scale), M, qw.K, qw.N, _ptr(qw.packed),
                                               _ptr(qw.scale), qw.scale.numel(), _qtype(qw.qtype), OUTS[out_mode],
                                               _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(),
                                               _stream(x.device)))
    return out


def qlinear_w8a8_dynamic(xq: torch.Tensor, x_scale: torch.Tensor, qw: QuantizedWeight, out_mode: str = "bf16",
                         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """W8A8 GEMM on per-token codes xq [M, K] with row scales x_scale fp32 [M]."""
    _require_gpu(xq, x_scale)
    if xq.dim() != 2 or xq.element_size() != 1 or xq.shape[1] != qw.K:
        raise ValueError(f"xq must be 1-byte codes [M, {qw.K}]")
    M = xq.shape[0]
    if x_scale.dtype != torch.float32 or x_scale.numel() != M:
        raise ValueError(f"x_scale must be fp32 [{M}]")
    if out is None:
        out = _w8a8_out(M, qw, out_mode, xq.device)
    nbytes = workspace_bytes("w8a8_dynamic", M, qw.K, qw.N, qw.qtype)
    ws = workspace if workspace is not None else _workspace(xq.device, nbytes)
    _check(lib().qlq_qlinear_w8a8_dynamic(_ptr(xq), _ptr(x_scale), M, qw.K, qw.N, _ptr(qw.packed),
                                          _ptr(qw.scale), qw.scale.numel(), _qtype(qw.qtype), OUTS[out_mode],
                                          _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(),
                                          _stream(xq.device)))
    return out


# ---------------------------------------------------------------------- routed Linear
LINEAR_SCHEMES = {"w8a16": 0, "w8a8_static": 1, "w8a8_dynamic": 3}


def linear_workspace_bytes(scheme: str, M: int, K: int, N: int, qtype: str) -> int:
    return int(lib().qlq_linear_workspace_bytes(LINEAR_SCHEMES[scheme], M, K, N, _qtype(qtype)))


def linear(scheme: str, x: torch.Tensor, qw: QuantizedWeight, input_scale: float = 1.0,
           bias: torch.Tensor | None = None, bf16_fallback_max_m: int = 0, out: torch.Tensor | None = None,
           workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Routed quantized Linear: bf16 x [M, K] -> bf16 y [M, N] (+ bf16 bias [N])."""
    _require_gpu(x)
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.shape[1] != qw.K:
        raise ValueError(f"x must be bf16 [M, {qw.K}]")
    if bias is not None:
        _require_gpu(bias)
        if bias.dtype != torch.bfloat16 or bias.numel() != qw.N:
            raise ValueError(f"bias must be bf16 [{qw.N}]")
    M = x.shape[0]
    if out is None:
        out = torch.empty((M, qw.N), dtype=torch.bfloat16, device=x.device)
    nbytes = linear_workspace_bytes(scheme, M, qw.K, qw.N, qw.qtype)
    ws = workspace if workspace is not None else _workspace(x.device, nbytes)
    _check(lib().qlq_linear(LINEAR_SCHEMES[scheme], _ptr(x), M, qw.K, qw.N, _ptr(qw.packed), _ptr(qw.scale),
                            qw.scale.numel(), _qtype(qw.qtype), float(input_scale), _ptr(bias),
                            int(bf16_fallback_max_m), _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(),
                            _stream(x.device)))
    return out


# ---------------------------------------------------------------------- KV cache
@dataclasses.dataclass
class QuantizedKV:
    """Mixed K-int8 / V-FP8 cache entries for [T, H, D] keys and values."""
    k_codes: torch.Tensor     # int8 [T, H, D]
    k_scales: torch.Tensor    # float16 [T, H, D / 32]
    v_codes: torch.Tensor     # uint8 e4m3fn bits [T, H, D]
    v_scales: torch.Tensor    # float16 [T, H]


def kv_quantize(k: torch.Tensor, v: torch.Tensor, out: QuantizedKV | None = None) -> QuantizedKV:
    """Quantize bf16 K and V [T, H, D] (D % 32 == 0) into cache entries."""
    _require_gpu(k, v)
    if k.dim() != 3 or k.shape != v.shape or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise ValueError("k and v must be bf16 [T, H, D] of the same shape")
    T, H, D = k.shape
    if out is None:
        out = QuantizedKV(torch.empty((T, H, D), dtype=torch.int8, device=k.device),
                          torch.empty((T, H, max(D // 32, 1)), dtype=torch.float16, device=k.device),
                          torch.empty((T, H, D), dtype=torch.uint8, device=k.device),
                          torch.empty((T, H), dtype=torch.float16, device=k.device))
    _check(lib().qlq_kv_quantize(_ptr(k), _ptr(v), T, H, D, _ptr(out.k_codes), _ptr(out.k_scales),
                                 _ptr(out.v_codes), _ptr(out.v_scales), _stream(k.device)))
    return out


def kv_dequantize(q: QuantizedKV, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None):
    """Cache entries -> bf16 (K, V) [T, H, D]."""
    _require_gpu(q.k_codes, q.k_scales, q.v_codes, q.v_scales)
    T, H, D = q.k_codes.shape
    if k_out is None:
        k_out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.k_codes.device)
    if v_out is None:
        v_out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.k_codes.device)
    _check(lib().qlq_kv_dequantize(_ptr(q.k_codes), _ptr(q.k_scales), _ptr(q.v_codes), _ptr(q.v_scales), T, H, D,
                                   _ptr(k_out), _ptr(v_out), _stream(q.k_codes.device)))
    return k_out, v_out


def kv_cache(slots: int, heads: int, head_dim: int, device: torch.device | str | None = None) -> QuantizedKV:
    """An empty cache of `slots` token entries (codes zero, scales one) for kv_append and kv_attention."""
    if slots < 1 or heads < 1 or head_dim < 32 or head_dim % 32 != 0:
        raise ValueError("slots and heads must be >= 1 and head_dim a multiple of 32")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return QuantizedKV(torch.zeros((slots, heads, head_dim), dtype=torch.int8, device=dev),
                       torch.ones((slots, heads, head_dim // 32), dtype=torch.float16, device=dev),
                       torch.zeros((slots, heads, head_dim), dtype=torch.uint8, device=dev),
                       torch.ones((slots, heads), dtype=torch.float16, device=dev))


# ---------------------------------------------------------------------- between the linears
# These calls take a few microseconds on the GPU, so what the host does before them counts: the raw
# handle of the current stream without a Stream object (0.1 against 1.9 us), outputs by empty_like,
# and every check of a tensor written out once (an attribute read and compared is 0.2 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _enqueue(dev: torch.device, fn, *args):
    """fn(*args, the current stream of dev), with dev as the current device."""
    index = dev.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(index))
    if status != 0:
        _check(status)


def _on(dev: torch.device, *ts):
    """Dense tensors (or None) on the GPU `dev`."""
    for t in ts:
        if t is not None:
            if t.device != dev:
                raise ValueError(f"all tensors must be on one GPU (got {t.device} and {dev})")
            if not t.is_contiguous():
                raise ValueError("qlq needs contiguous (row-major) tensors")


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _norm_inputs(x, weight, residual, residual_out):
    if not x.is_cuda:
        raise ValueError("qlq operates on GPU tensors only")
    bf = torch.bfloat16
    shape = x.shape
    if len(shape) != 2 or x.dtype != bf:
        raise ValueError("x must be a 2-D bf16 tensor")
    if weight.dtype != bf or weight.shape != shape[1:]:
        raise ValueError(f"weight must be bf16 [{shape[1]}]")
    dev = x.device
    if not x.is_contiguous() or weight.device != dev or not weight.is_contiguous():
        _on(dev, x, weight)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return None
    if residual.dtype != bf or residual.shape != shape or (
            residual_out is not None and (residual_out.dtype != bf or residual_out.shape != shape)):
        raise ValueError(f"residual and residual_out must be bf16 {list(shape)}")
    if residual_out is not None:
        _on(dev, residual, residual_out)
        return residual_out
    if residual.device != dev or not residual.is_contiguous():
        _on(dev, residual)
    return torch.empty_like(x)


def _norm_codes(x, qtype, out):
    if out is None:
        return torch.empty_like(x, dtype=code_dtype(qtype))
    if out.element_size() != 1 or out.shape != x.shape:
        raise ValueError(f"out must be 1-byte codes {list(x.shape)}")
    _on(x.device, out)
    return out


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
             out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None):
    """RMS norm of x [M, K] bf16 rows: y bf16 [M, K]; with a residual, (y, h) where h = bf16(x + residual) and
    y is the norm of the unrounded sum.  out and residual_out may be x or residual."""
    residual_out = _norm_inputs(x, weight, residual, residual_out)
    if out is None:
        out = torch.empty_like(x)
    elif out.dtype != torch.bfloat16 or out.shape != x.shape:
        raise ValueError(f"out must be bf16 {list(x.shape)}")
    else:
        _on(x.device, out)
    _enqueue(x.device, lib().qlq_rms_norm, x.data_ptr(), _addr(residual), weight.data_ptr(), x.shape[0], x.shape[1],
             eps, out.data_ptr(), _addr(residual_out))
    return out if residual is None else (out, residual_out)


def rms_norm_quant_static(x: torch.Tensor, weight: torch.Tensor, input_scale: float, qtype: str, eps: float = 1e-6,
                          residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                          residual_out: torch.Tensor | None = None):
    """rms_norm straight to the codes of a static W8A8 linear's input: xq [M, K]; with a residual, (xq, h)."""
    q = _qtype(qtype)
    residual_out = _norm_inputs(x, weight, residual, residual_out)
    out = _norm_codes(x, qtype, out)
    _enqueue(x.device, lib().qlq_rms_norm_quant_static, x.data_ptr(), _addr(residual), weight.data_ptr(), x.shape[0],
             x.shape[1], eps, float(input_scale), q, out.data_ptr(), _addr(residual_out))
    return out if residual is None else (out, residual_out)


def rms_norm_quant_dynamic(x: torch.Tensor, weight: torch.Tensor, qtype: str, eps: float = 1e-6,
                           residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                           x_scale: torch.Tensor | None = None, residual_out: torch.Tensor | None = None):
    """rms_norm straight to per-token codes and scales (qlinear_w8a8_dynamic's input): (xq [M, K], x_scale fp32
    [M]); with a residual, (xq, x_scale, h)."""
    q = _qtype(qtype)
    residual_out = _norm_inputs(x, weight, residual, residual_out)
    out = _norm_codes(x, qtype, out)
    if x_scale is None:
        x_scale = x.new_empty(x.shape[0], dtype=torch.float32)
    elif x_scale.dtype != torch.float32 or x_scale.numel() != x.shape[0]:
        raise ValueError(f"x_scale must be fp32 [{x.shape[0]}]")
    else:
        _on(x.device, x_scale)
    _enqueue(x.device, lib().qlq_rms_norm_quant_dynamic, x.data_ptr(), _addr(residual), weight.data_ptr(), x.shape[0],
             x.shape[1], eps, q, out.data_ptr(), x_scale.data_ptr(), _addr(residual_out))
    return (out, x_scale) if residual is None else (out, x_scale, residual_out)


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: dict | None = None,
                  device: torch.device | str | None = None):
    """(inv_freq fp64 [rotary_dim / 2] on the GPU, attention_factor): rotary frequencies base^(-2i / rotary_dim),
    scaled for long contexts by `scaling`:
      None
      {"type": "linear", "factor": f}      every frequency / f
      {"type": "ntk", "factor": f}         base * f^(rotary_dim / (rotary_dim - 2))
      {"type": "yarn", "factor": f, "original_max_positions": n, "beta_fast": 32, "beta_slow": 1,
       "attention_factor": 0.1 ln f + 1}   frequencies / f below beta_slow turns over n positions, unchanged above
                                           beta_fast, a ramp between (by channel)
      {"type": "llama3", "factor": f, "original_max_positions": n, "low_freq_factor": 1, "high_freq_factor": 4}
                                           / f for wavelengths above n / low, unchanged below n / high, blended
                                           between (by wavelength)"""
    R = int(rotary_dim)
    if R < 2 or R % 2 != 0:
        raise ValueError("rotary_dim must be even and >= 2")
    if not (math.isfinite(base) and base > 1.0):
        raise ValueError("base must be finite and > 1")
    kind, factor, extra = None, 1.0, {}
    if scaling is not None:
        extra = dict(scaling)
        kind = extra.pop("type", None)
        known = {"linear": set(), "ntk": set(), "yarn": {"original_max_positions", "beta_fast", "beta_slow",
                                                         "attention_factor"},
                 "llama3": {"original_max_positions", "low_freq_factor", "high_freq_factor"}}
        if kind not in known:
            raise ValueError(f"scaling type must be one of {sorted(known)}")
        factor = float(extra.pop("factor", 1.0))
        if not (math.isfinite(factor) and factor > 0.0):
            raise ValueError("scaling factor must be finite and > 0")
        if set(extra) - known[kind]:
            raise ValueError(f"unknown {kind} scaling keys {sorted(set(extra) - known[kind])}")
        if kind in ("yarn", "llama3") and not extra.get("original_max_positions", 0) > 0:
            raise ValueError(f"{kind} scaling needs original_max_positions")
    if kind == "ntk":
        if R == 2:
            raise ValueError("ntk scaling needs rotary_dim > 2")
        base = base * factor ** (R / (R - 2))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    attention_factor = 1.0
    if kind == "linear":
        f = [v / factor for v in f]
    elif kind == "yarn":
        n = float(extra["original_max_positions"])

        def channel(turns):      # the (fractional) pair index that makes `turns` turns over n positions
            return R * math.log(n / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        lo = max(math.floor(channel(float(extra.get("beta_fast", 32.0)))), 0)
        hi = min(math.ceil(channel(float(extra.get("beta_slow", 1.0)))), R - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(R // 2)]
        f = [v / factor * r + v * (1.0 - r) for v, r in zip(f, ramp)]
        attention_factor = float(extra.get("attention_factor", 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0))
    elif kind == "llama3":
        n = float(extra["original_max_positions"])
        low, high = float(extra.get("low_freq_factor", 1.0)), float(extra.get("high_freq_factor", 4.0))
        if not 0.0 < low < high:
            raise ValueError("llama3 scaling needs 0 < low_freq_factor < high_freq_factor")
        smooth = [min(max((n * v / (2.0 * math.pi) - low) / (high - low), 0.0), 1.0) for v in f]
        f = [v / factor * (1.0 - s) + v * s for v, s in zip(f, smooth)]
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return torch.tensor(f, dtype=torch.float64, device=dev), attention_factor


def _token_rows(t: torch.Tensor, name: str) -> int:
    """Token stride of a bf16 GPU tensor [T, H, D] whose heads and channels are dense."""
    if not t.is_cuda:
        raise ValueError("qlq operates on GPU tensors only")
    if t.dim() != 3 or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bf16 [T, H, D]")
    st, sh, sd = t.stride()
    T, H, D = t.shape
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError(f"{name} must be dense in its heads and channels (only the token stride is free)")
    return st if T > 1 else H * D


def _indices(t: torch.Tensor, n: int, dev: torch.device, name: str) -> int:
    """1 for int64, 0 for int32 indices [n] on dev."""
    dtype = t.dtype
    if (dtype != torch.int64 and dtype != torch.int32) or t.shape != (n,):
        raise ValueError(f"{name} must be int32 or int64 [{n}]")
    if t.device != dev or not t.is_contiguous():
        _on(dev, t)
    return 1 if dtype == torch.int64 else 0


def _frequencies(inv_freq: torch.Tensor, dev: torch.device) -> int:
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be fp64 [rotary_dim / 2] (rope_inv_freq)")
    _on(dev, inv_freq)
    return 2 * inv_freq.shape[0]


def _cache_entries(c: QuantizedKV, H: int, D: int, dev: torch.device) -> int:
    """Slots of a cache for H heads of D channels."""
    kc, ks, vc, vs = c.k_codes, c.k_scales, c.v_codes, c.v_scales
    if D % 32 != 0:
        raise ValueError("head_dim must be a multiple of 32")
    shape = kc.shape
    P = shape[0]
    if shape != (P, H, D) or vc.shape != shape or ks.shape != (P, H, D // 32) or vs.shape != (P, H):
        raise ValueError(f"the cache must hold [slots, {H}, {D}] entries")
    if kc.element_size() != 1 or vc.element_size() != 1 or ks.dtype != torch.float16 or vs.dtype != torch.float16:
        raise ValueError("the cache must hold 1-byte codes and float16 scales")
    if not (kc.device == ks.device == vc.device == vs.device == dev and kc.is_contiguous() and ks.is_contiguous()
            and vc.is_contiguous() and vs.is_contiguous()):
        _on(dev, kc, ks, vc, vs)
    return P


def rope(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, attention_factor: float = 1.0,
         interleaved: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotary positions on the first 2 * len(inv_freq) channels of x [T, H, D] bf16 (pairs (i, i + R/2), or (2i,
    2i+1) interleaved); the token stride of x is free.  out may be x."""
    xs = _token_rows(x, "x")
    T, H, D = x.shape
    R = _frequencies(inv_freq, x.device)
    p64 = _indices(positions, T, x.device, "positions")
    if out is None:
        out, os_ = torch.empty_like(x, memory_format=torch.contiguous_format), H * D
    else:
        os_ = _token_rows(out, "out")
        if out.shape != x.shape or out.device != x.device:
            raise ValueError(f"out must be bf16 {list(x.shape)} on {x.device}")
    _enqueue(x.device, lib().qlq_rope, x.data_ptr(), xs, T, H, D, positions.data_ptr(), p64, inv_freq.data_ptr(), R,
             float(attention_factor), int(interleaved), out.data_ptr(), os_)
    return out


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: QuantizedKV, slots: torch.Tensor) -> QuantizedKV:
    """Quantize k, v [T, H, D] bf16 (as kv_quantize; token strides free) into cache entries slots [T].  A slot
    outside the cache (padding: -1) is not written; slots must not repeat.  Returns the cache."""
    ks, vs = _token_rows(k, "k"), _token_rows(v, "v")
    if k.shape != v.shape or k.device != v.device:
        raise ValueError("k and v must have the same shape and device")
    T, H, D = k.shape
    P = _cache_entries(cache, H, D, k.device)
    s64 = _indices(slots, T, k.device, "slots")
    _enqueue(k.device, lib().qlq_kv_append, k.data_ptr(), ks, v.data_ptr(), vs, T, H, D, slots.data_ptr(), s64, P,
             cache.k_codes.data_ptr(), cache.k_scales.data_ptr(), cache.v_codes.data_ptr(), cache.v_scales.data_ptr())
    return cache


def rope_kv_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
                   cache: QuantizedKV, slots: torch.Tensor, attention_factor: float = 1.0, interleaved: bool = False,
                   q_out: torch.Tensor | None = None) -> torch.Tensor:
    """rope of q [T, Hq, D] and k [T, Hk, D], and kv_append of the rotated k and of v, in one kernel.  q, k and v
    may be views of one projection's output.  Returns the rotated q (q_out may be q)."""
    qs, ks, vs = _token_rows(q, "q"), _token_rows(k, "k"), _token_rows(v, "v")
    T, Hq, D = q.shape
    dev = q.device
    if k.shape != v.shape or k.shape[0] != T or k.shape[2] != D or k.device != dev or v.device != dev:
        raise ValueError("k and v must be [T, Hk, D] with q's T, D and device")
    Hk = k.shape[1]
    P = _cache_entries(cache, Hk, D, dev)
    R = _frequencies(inv_freq, dev)
    p64, s64 = _indices(positions, T, dev, "positions"), _indices(slots, T, dev, "slots")
    if q_out is None:
        q_out, os_ = torch.empty_like(q, memory_format=torch.contiguous_format), Hq * D
    else:
        os_ = _token_rows(q_out, "q_out")
        if q_out.shape != q.shape or q_out.device != dev:
            raise ValueError(f"q_out must be bf16 {list(q.shape)} on {dev}")
    _enqueue(dev, lib().qlq_rope_kv_append, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, Hq, Hk, D,
             positions.data_ptr(), p64, inv_freq.data_ptr(), R, float(attention_factor), int(interleaved),
             slots.data_ptr(), s64, P, cache.k_codes.data_ptr(), cache.k_scales.data_ptr(), cache.v_codes.data_ptr(),
             cache.v_scales.data_ptr(), q_out.data_ptr(), os_)
    return q_out


def kv_gather(cache: QuantizedKV, slots: torch.Tensor, k_out: torch.Tensor | None = None,
              v_out: torch.Tensor | None = None):
    """Cache entries slots [n] as dense bf16 (K, V) [n, H, D]; zeros for a slot outside the cache."""
    dev = cache.k_codes.device
    if not cache.k_codes.is_cuda:
        raise ValueError("qlq operates on GPU tensors only")
    _, H, D = cache.k_codes.shape
    P = _cache_entries(cache, H, D, dev)
    n = slots.shape[0] if slots.dim() == 1 else -1
    s64 = _indices(slots, n, dev, "slots")
    outs = []
    for t in (k_out, v_out):
        if t is None:
            t = torch.empty_like(outs[0]) if outs else torch.empty(n, H, D, dtype=torch.bfloat16, device=dev)
        elif t.dtype != torch.bfloat16 or t.shape != (n, H, D):
            raise ValueError(f"k_out and v_out must be bf16 [{n}, {H}, {D}]")
        else:
            _on(dev, t)
        outs.append(t)
    _enqueue(dev, lib().qlq_kv_gather, cache.k_codes.data_ptr(), cache.k_scales.data_ptr(), cache.v_codes.data_ptr(),
             cache.v_scales.data_ptr(), P, H, D, slots.data_ptr(), s64, n, outs[0].data_ptr(), outs[1].data_ptr())
    return outs[0], outs[1]


@functools.lru_cache(maxsize=1024)
def kv_attention_workspace_bytes(T: int, B: int, Hq: int, Hk: int, D: int, one_each: bool = True) -> int:
    """Workspace of kv_attention for T query tokens of B sequences (one_each: without q_start)."""
    return int(lib().qlq_kv_attention_workspace_bytes(T, B, Hq, Hk, D, int(one_each)))


_ATTENTION_COUNTER_BYTES = 262144
_ATTENTION_STREAMS = 40                  # workspaces kept: torch's 32 pooled streams, the default one, some of a user's
_attention_workspaces: dict = {}


def _attention_workspace(dev: torch.device, nbytes: int) -> torch.Tensor:
    """A workspace of this stream with its counters zeroed, grown on demand; inside a graph capture, one of the
    graph's own (its zero fill is recorded with it), so that graphs and streams never share one.  The oldest
    goes when there are many (its memory returns to the allocator's pool of its stream, in that stream's order)."""
    capturing = torch.cuda.is_current_stream_capturing()
    key = (dev.index, _raw_stream(dev.index))
    ws = None if capturing else _attention_workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        ws[:_ATTENTION_COUNTER_BYTES].zero_()
        if not capturing:
            with _lock:
                _attention_workspaces.pop(key, None)
                while len(_attention_workspaces) >= _ATTENTION_STREAMS:
                    del _attention_workspaces[next(iter(_attention_workspaces))]
                _attention_workspaces[key] = ws
    return ws


def kv_attention(q: torch.Tensor, cache: QuantizedKV, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 page_size: int, q_start: torch.Tensor | None = None, scale: float | None = None, causal: bool = True,
                 window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of q [T, Hq, D] bf16 over a paged cache (kv_append): out bf16 [T, Hq, D].

    block_table int32 [B, pages] holds each sequence's page numbers (token t is cache entry
    block_table[b][t // page_size] * page_size + t % page_size; page_size a power of two from 16), seq_lens int32
    [B] its cached tokens.  Without q_start, row b of q is the last token of sequence b; with q_start int32 [B + 1],
    rows q_start[b] .. q_start[b+1]-1 are its last tokens.  A query sees the tokens up to its own (causal), and no
    more than `window` of them if that is not 0.  scale defaults to D^-0.5; lse fp32 [T, Hq], if given, receives log
    sum exp of the scaled scores.  Rows that see nothing give zeros (lse -inf); rows of no sequence are left as they
    were.
    The lengths stay on the device: nothing here waits for them.  One kernel is chosen for all rows by their average
    per sequence, so prompts and single tokens are faster in a call each.

    workspace: uint8, zeros before its first use, of kv_attention_workspace_bytes(T, B, Hq, Hk, D, q_start is None)
    bytes or more, for this function's calls on one stream at a time.  Without it, one is kept per stream; in a graph
    capture every call gets its own and records its zero fill (2 us), which one workspace for all of a graph's
    calls saves."""
    qs = _token_rows(q, "q")
    T, Hq, D = q.shape
    dev = q.device
    if cache.k_codes.dim() != 3:
        raise ValueError("the cache must hold [slots, heads, head_dim] entries")
    Hk = cache.k_codes.shape[1]
    P = _cache_entries(cache, Hk, D, dev)
    if block_table.dim() != 2 or block_table.dtype != torch.int32:
        raise ValueError("block_table must be int32 [B, pages]")
    B = block_table.shape[0]
    if seq_lens.dtype != torch.int32 or seq_lens.shape != (B,):
        raise ValueError(f"seq_lens must be int32 [{B}]")
    if q_start is not None and (q_start.dtype != torch.int32 or q_start.shape != (B + 1,)):
        raise ValueError(f"q_start must be int32 [{B + 1}]")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif out.dtype != torch.bfloat16 or out.shape != q.shape:
        raise ValueError(f"out must be bf16 {list(q.shape)}")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, Hq)):
        raise ValueError(f"lse must be fp32 [{T}, {Hq}]")
    _on(dev, block_table, seq_lens, q_start, out, lse, workspace)
    if workspace is None:
        workspace = _attention_workspace(dev, kv_attention_workspace_bytes(T, B, Hq, Hk, D, q_start is None))
    _enqueue(dev, lib().qlq_kv_attention, q.data_ptr(), qs, T, B, Hq, Hk, D, cache.k_codes.data_ptr(),
             cache.k_scales.data_ptr(), cache.v_codes.data_ptr(), cache.v_scales.data_ptr(), P,
             block_table.data_ptr(), block_table.shape[1], page_size, seq_lens.data_ptr(), _addr(q_start),
             D ** -0.5 if scale is None else float(scale), int(causal), int(window), out.data_ptr(), _addr(lse),
             workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out
