"""Python binding of libdbf, the MI355X DBF linear-forward library.

Double Binary Factorization stores a weight matrix as
W = diag(a) A diag(mid) B diag(b) with +/-1 factors A (n x k), B (k x m) and
fp16 scale vectors ("Addition is almost all you need: Compressing large
language models with double binary factorization", gist.science technical
summary, §2.1).  The library evaluates Y = X W^T on the GPU without forming W.

This module only marshals arguments to the C ABI declared in include/dbf.h:
every step of the forward runs in the library's HIP kernels.  PyTorch is
used for device memory and the current stream, nothing else.  If the shared
library has not been built the first call raises a RuntimeError; there is no
fallback of any kind.
"""

from __future__ import annotations

import ctypes
import os
from typing import Dict, NamedTuple, Optional

import numpy as np

__all__ = [
    "DBF_OK", "DBF_ERR_INVALID_ARG", "DBF_ERR_SHAPE", "DBF_ERR_OOM", "DBF_ERR_HIP", "DBF_ERR_UNSUPPORTED",
    "DBF_PATH_AUTO", "DBF_PATH_DECODE", "DBF_PATH_PREFILL", "DBF_PATH_DECODE_TABLE", "DBF_PATH_DECODE_EXACT",
    "EXPORTED_SYMBOLS",
    "DbfError", "lib", "library_path",
    "dbf_pack", "dbf_linear_forward", "dbf_linear_forward_ex", "dbf_free", "dbf_get_info",
    "dbf_status_string", "dbf_pack_signs", "dbf_layout_signs", "dbf_layout_words", "dbf_layout_signs_dec",
    "dbf_layout_words_dec",
    "dbf_timing_enable", "dbf_timing_read", "Layer", "dbf_linear_forward_group", "forward_group",
    "dbf_pack_ex", "dbf_linear_backward_data", "dbf_linear_backward", "DBF_PACK_BACKWARD", "dbf_bqq_pack",
    "dbf_factorize", "factorize", "dbf_linear_forward_noalloc", "dbf_bqq_pack_grouped",
    "DBF_TYPE_F16", "DBF_TYPE_BF16", "DBF_TYPE_F32", "DBF_TYPE_E4M3", "DBF_TYPE_E2M1", "MxTensor", "mx_quantize",
    "dbf_mx_pack", "dbf_mx_forward_plan", "dbf_mx_backward_plan", "rms_norm", "RmsNormOutput", "rms_norm_backward", "norm_forward_group",
    "RowGroups", "group_rows", "dbf_experts_pack", "dbf_experts_forward_plan", "dbf_experts_backward_plan", "Experts", "Adapters", "AdapterOutput",
]

DBF_OK = 0
DBF_ERR_INVALID_ARG = 1
DBF_ERR_SHAPE = 2
DBF_ERR_OOM = 3
DBF_ERR_HIP = 4
DBF_ERR_UNSUPPORTED = 5

DBF_PATH_AUTO = 0
DBF_PATH_DECODE = 1
DBF_PATH_PREFILL = 2
DBF_PATH_DECODE_TABLE = 3
DBF_PATH_DECODE_EXACT = 4

DBF_PACK_BACKWARD = 1

DBF_TYPE_F16 = 0
DBF_TYPE_BF16 = 1
DBF_TYPE_F32 = 2
DBF_TYPE_E4M3 = 3
DBF_TYPE_E2M1 = 4

DECODE_MAX_BATCH = 16

EXPORTED_SYMBOLS = (
    "dbf_pack", "dbf_pack_ex", "dbf_linear_forward", "dbf_linear_forward_ex", "dbf_linear_forward_group",
    "dbf_linear_backward_data", "dbf_linear_backward", "dbf_free", "dbf_get_info", "dbf_status_string",
    "dbf_pack_signs", "dbf_layout_signs", "dbf_layout_words", "dbf_layout_signs_dec", "dbf_layout_words_dec",
    "dbf_timing_enable", "dbf_timing_read", "dbf_bqq_pack", "dbf_factorize", "dbf_linear_forward_noalloc",
    "dbf_bqq_pack_grouped", "dbf_mx_code_bytes", "dbf_mx_scale_bytes", "dbf_mx_quantize", "dbf_mx_dequantize",
    "dbf_mx_pack", "dbf_mx_forward", "dbf_mx_forward_group", "dbf_mx_backward_data", "dbf_mx_forward_plan",
    "dbf_mx_backward_plan", "dbf_rms_norm", "dbf_rms_norm_backward_workspace", "dbf_rms_norm_backward",
    "dbf_group_rows_workspace", "dbf_group_rows", "dbf_experts_pack", "dbf_experts_forward",
    "dbf_experts_backward_data", "dbf_experts_forward_plan", "dbf_experts_backward_plan", "dbf_adapter_workspace", "dbf_adapter_forward", "dbf_adapter_backward_workspace",
    "dbf_adapter_backward",
)

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libdbf.so")
_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return _LIB_PATH


class DbfError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dbf_status_string(status)} (status {status})")


class _Info(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int32), ("m", ctypes.c_int32), ("k", ctypes.c_int32),
        ("n_pad", ctypes.c_int32), ("m_pad", ctypes.c_int32), ("k_pad", ctypes.c_int32),
        ("max_batch", ctypes.c_int32), ("device", ctypes.c_int32),
        ("packed_bytes", ctypes.c_size_t), ("scale_bytes", ctypes.c_size_t),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class _KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double)]


def lib() -> ctypes.CDLL:
    """Load libdbf.so (once).  Raises RuntimeError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is missing: build it with `python -m dbf_linear_fwd_amd.build` "
            "(the DBF forward has no non-HIP implementation)")
    # PyTorch brings a HIP runtime of its own.  Loaded first, it serves the
    # library too; loaded after the library, the process has two, and calls on
    # PyTorch's memory and streams fail.
    try:
        import torch  # noqa: F401
    except (ImportError, OSError):  # (none, or one that does not load here)
        pass
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    L.dbf_pack.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, i32, ctypes.POINTER(vp)]
    L.dbf_pack.restype = ctypes.c_int
    L.dbf_linear_forward.argtypes = [vp, vp, vp, i32, vp]
    L.dbf_linear_forward.restype = ctypes.c_int
    L.dbf_linear_forward_ex.argtypes = [vp, vp, vp, i32, i32, vp]
    L.dbf_linear_forward_ex.restype = ctypes.c_int
    L.dbf_linear_forward_noalloc.argtypes = [vp, vp, vp, i32, vp]
    L.dbf_linear_forward_noalloc.restype = ctypes.c_int
    L.dbf_pack_ex.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, i32, i32, ctypes.POINTER(vp)]
    L.dbf_pack_ex.restype = ctypes.c_int
    L.dbf_bqq_pack.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, ctypes.c_uint16, i32, ctypes.POINTER(vp)]
    L.dbf_bqq_pack.restype = ctypes.c_int
    L.dbf_bqq_pack_grouped.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, i32, ctypes.POINTER(vp)]
    L.dbf_bqq_pack_grouped.restype = ctypes.c_int
    L.dbf_factorize.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, ctypes.c_float, i32, i32, i32,
                                vp, vp, vp, vp, vp, vp, vp]
    L.dbf_factorize.restype = ctypes.c_int
    L.dbf_linear_backward_data.argtypes = [vp, vp, vp, i32, vp]
    L.dbf_linear_backward_data.restype = ctypes.c_int
    L.dbf_linear_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp]
    L.dbf_linear_backward.restype = ctypes.c_int
    L.dbf_linear_forward_group.argtypes = [ctypes.POINTER(vp), i32, vp, ctypes.POINTER(vp), i32, vp]
    L.dbf_linear_forward_group.restype = ctypes.c_int
    L.dbf_mx_code_bytes.argtypes = [i32, i32]
    L.dbf_mx_code_bytes.restype = sz
    L.dbf_mx_scale_bytes.argtypes = [i32]
    L.dbf_mx_scale_bytes.restype = sz
    L.dbf_mx_quantize.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
    L.dbf_mx_quantize.restype = ctypes.c_int
    L.dbf_mx_dequantize.argtypes = [vp, vp, i32, i32, i32, vp, i32, vp]
    L.dbf_mx_dequantize.restype = ctypes.c_int
    L.dbf_mx_pack.argtypes = [i32, i32, vp, vp, i32, i32, vp, ctypes.POINTER(vp)]
    L.dbf_mx_pack.restype = ctypes.c_int
    L.dbf_mx_forward.argtypes = [vp, vp, i32, vp, vp, i32, i32, vp]
    L.dbf_mx_forward.restype = ctypes.c_int
    L.dbf_mx_forward_group.argtypes = [ctypes.POINTER(vp), i32, vp, i32, vp, ctypes.POINTER(vp), i32, i32, vp]
    L.dbf_mx_forward_group.restype = ctypes.c_int
    L.dbf_mx_backward_data.argtypes = [vp, vp, vp, i32, i32, vp]
    L.dbf_mx_backward_data.restype = ctypes.c_int
    L.dbf_mx_forward_plan.argtypes = [i32, i32, i32, i32, ctypes.POINTER(i32)]
    L.dbf_mx_forward_plan.restype = ctypes.c_int
    L.dbf_mx_backward_plan.argtypes = [i32, i32, i32, ctypes.POINTER(i32)]
    L.dbf_mx_backward_plan.restype = ctypes.c_int
    L.dbf_rms_norm.argtypes = [vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, vp, vp, i32, vp, vp, vp]
    L.dbf_rms_norm.restype = ctypes.c_int
    L.dbf_rms_norm_backward_workspace.argtypes = [i32, i32]
    L.dbf_rms_norm_backward_workspace.restype = sz
    L.dbf_rms_norm_backward.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, sz, vp]
    L.dbf_rms_norm_backward.restype = ctypes.c_int
    L.dbf_group_rows_workspace.argtypes = [i32, i32]
    L.dbf_group_rows_workspace.restype = sz
    L.dbf_group_rows.argtypes = [vp, i32, i32, i32, vp, vp, vp, sz, vp]
    L.dbf_group_rows.restype = ctypes.c_int
    L.dbf_experts_pack.argtypes = [i32, i32, i32, vp, vp, i32, i32, vp, ctypes.POINTER(vp)]
    L.dbf_experts_pack.restype = ctypes.c_int
    L.dbf_experts_forward.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, vp, i32, vp]
    L.dbf_experts_forward.restype = ctypes.c_int
    L.dbf_experts_backward_data.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, vp, vp]
    L.dbf_experts_backward_data.restype = ctypes.c_int
    L.dbf_experts_forward_plan.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(i32)]
    L.dbf_experts_forward_plan.restype = ctypes.c_int
    L.dbf_experts_backward_plan.argtypes = [i32, i32, i32, i32, ctypes.POINTER(i32)]
    L.dbf_experts_backward_plan.restype = ctypes.c_int
    for name in ("dbf_adapter_workspace", "dbf_adapter_backward_workspace"):
        getattr(L, name).argtypes = [i32, i32, i32, i32, i32]
        getattr(L, name).restype = sz
    L.dbf_adapter_forward.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, sz, vp]
    L.dbf_adapter_forward.restype = ctypes.c_int
    L.dbf_adapter_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp,
                                       vp, sz, vp]
    L.dbf_adapter_backward.restype = ctypes.c_int
    L.dbf_free.argtypes = [vp]
    L.dbf_free.restype = None
    L.dbf_get_info.argtypes = [vp, ctypes.POINTER(_Info)]
    L.dbf_get_info.restype = ctypes.c_int
    L.dbf_status_string.argtypes = [ctypes.c_int]
    L.dbf_status_string.restype = ctypes.c_char_p
    L.dbf_pack_signs.argtypes = [vp, i32, i32, vp, i32]
    L.dbf_pack_signs.restype = ctypes.c_int
    L.dbf_layout_signs.argtypes = [vp, i32, i32, vp]
    L.dbf_layout_signs.restype = ctypes.c_int
    L.dbf_layout_words.argtypes = [i32, i32]
    L.dbf_layout_words.restype = sz
    L.dbf_layout_signs_dec.argtypes = [vp, i32, i32, i32, i32, i32, vp]
    L.dbf_layout_signs_dec.restype = ctypes.c_int
    L.dbf_layout_words_dec.argtypes = [i32, i32]
    L.dbf_layout_words_dec.restype = sz
    L.dbf_timing_enable.argtypes = [vp, i32]
    L.dbf_timing_enable.restype = ctypes.c_int
    L.dbf_timing_read.argtypes = [vp, ctypes.POINTER(_KernelTime), i32, ctypes.POINTER(i32)]
    L.dbf_timing_read.restype = ctypes.c_int
    _lib = L
    return L


def _check(status: int, where: str) -> None:
    if status != DBF_OK:
        raise DbfError(status, where)


def _ptr(arr: np.ndarray) -> int:
    return arr.ctypes.data


def dbf_status_string(status: int) -> str:
    return lib().dbf_status_string(int(status)).decode()


def _as_signs(S) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(S), dtype=np.int8)


def _as_half_bits(v) -> np.ndarray:
    v = np.asarray(v)
    if v.dtype == np.uint16:
        return np.ascontiguousarray(v)
    return np.ascontiguousarray(v.astype(np.float16)).view(np.uint16)


def dbf_pack(n: int, m: int, k: int, A_signs, B_signs, a, mid, b, max_batch: int, flags: int = 0) -> int:
    """Build a layer handle (see dbf_pack / dbf_pack_ex in include/dbf.h).  Returns the handle as an int."""
    A = _as_signs(A_signs)
    B = _as_signs(B_signs)
    if A.size != n * k or B.size != k * m:
        raise ValueError("A must hold n*k and B k*m entries")
    a16, mid16, b16 = _as_half_bits(a), _as_half_bits(mid), _as_half_bits(b)
    if a16.size != n or mid16.size != k or b16.size != m:
        raise ValueError("a, mid, b must have lengths n, k, m")
    h = ctypes.c_void_p()
    if flags:
        st = lib().dbf_pack_ex(n, m, k, _ptr(A), _ptr(B), _ptr(a16), _ptr(mid16), _ptr(b16), max_batch, flags,
                               ctypes.byref(h))
    else:
        st = lib().dbf_pack(n, m, k, _ptr(A), _ptr(B), _ptr(a16), _ptr(mid16), _ptr(b16), max_batch,
                            ctypes.byref(h))
    _check(st, "dbf_pack")
    return h.value


def dbf_bqq_pack(n: int, m: int, d: int, p: int, Y, Z, r, s, t, u, max_batch: int) -> int:
    """Handle of a BQQ-form layer (see dbf_bqq_pack in include/dbf.h): Y (p, n, d) and
    Z (p, d, m) of 0/1, fp16 scalars r, s, t (p each) and u."""
    Y8 = np.ascontiguousarray(np.asarray(Y), dtype=np.uint8)
    Z8 = np.ascontiguousarray(np.asarray(Z), dtype=np.uint8)
    if Y8.size != p * n * d or Z8.size != p * d * m:
        raise ValueError("Y must hold p*n*d and Z p*d*m entries")
    r16, s16, t16 = _as_half_bits(r), _as_half_bits(s), _as_half_bits(t)
    if r16.size != p or s16.size != p or t16.size != p:
        raise ValueError("r, s, t must have p entries")
    u16 = int(_as_half_bits(np.asarray([u]))[0])
    h = ctypes.c_void_p()
    _check(lib().dbf_bqq_pack(n, m, d, p, _ptr(Y8), _ptr(Z8), _ptr(r16), _ptr(s16), _ptr(t16), u16, max_batch,
                              ctypes.byref(h)), "dbf_bqq_pack")
    return h.value


def dbf_bqq_pack_grouped(n: int, m: int, d: int, p: int, group: int, Y, Z, r, s, t, u, max_batch: int) -> int:
    """Handle of a BQQ-form layer with group-wise scalars (see dbf_bqq_pack_grouped in
    include/dbf.h): Y (p, n, d) and Z (p, d, m) of 0/1, fp16 r, s, t (p, ngroups) and u
    (ngroups,), ngroups = ceil(m / group)."""
    Y8 = np.ascontiguousarray(np.asarray(Y), dtype=np.uint8)
    Z8 = np.ascontiguousarray(np.asarray(Z), dtype=np.uint8)
    if Y8.size != p * n * d or Z8.size != p * d * m:
        raise ValueError("Y must hold p*n*d and Z p*d*m entries")
    if group < 1:
        raise ValueError("group must be positive")
    ng = -(-m // group)
    r16, s16, t16, u16 = _as_half_bits(r), _as_half_bits(s), _as_half_bits(t), _as_half_bits(u)
    if r16.size != p * ng or s16.size != p * ng or t16.size != p * ng or u16.size != ng:
        raise ValueError(f"r, s, t must have p * ngroups = {p * ng} entries and u ngroups = {ng}")
    h = ctypes.c_void_p()
    _check(lib().dbf_bqq_pack_grouped(n, m, d, p, group, _ptr(Y8), _ptr(Z8), _ptr(r16), _ptr(s16), _ptr(t16),
                                      _ptr(u16), max_batch, ctypes.byref(h)), "dbf_bqq_pack_grouped")
    return h.value


def dbf_factorize(W_ptr: int, n: int, m: int, k: int, U0_ptr: int, V0_ptr: int, dout_ptr: int, din_ptr: int,
                  rho_rel: float, outer: int, inner: int, power_iters: int, A_ptr: int, B_ptr: int, a_ptr: int,
                  mid_ptr: int, b_ptr: int, err_ptr: int, stream: int = 0) -> None:
    _check(lib().dbf_factorize(W_ptr, n, m, k, U0_ptr, V0_ptr, dout_ptr or None, din_ptr or None, rho_rel, outer,
                               inner, power_iters, A_ptr, B_ptr, a_ptr, mid_ptr, b_ptr, err_ptr or None, stream),
           "dbf_factorize")


def factorize(W, k: int, U0, V0, rho_rel: float = 1.0, outer: int = 2, inner: int = 4, power_iters: int = 8,
              d_out=None, d_in=None):
    """DBF factors of W (CUDA float32 tensor, n x m) from the starting factors
    U0 (n x k) and V0 (k x m): returns (A, B, a, mid, b, err) as CUDA tensors
    (int8 +/-1, int8 +/-1, float16 x 3, float32 [outer])."""
    import torch

    def dev32(t, shape, what):
        if t is None:
            return None
        if t.dtype != torch.float32 or not t.is_cuda or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous CUDA float32 tensor of shape {shape}")
        return t
    n, m = W.shape
    dev32(W, (n, m), "W")
    dev32(U0, (n, k), "U0")
    dev32(V0, (k, m), "V0")
    dev32(d_out, (n,), "d_out")
    dev32(d_in, (m,), "d_in")
    dev = W.device
    A = torch.empty((n, k), dtype=torch.int8, device=dev)
    B = torch.empty((k, m), dtype=torch.int8, device=dev)
    a = torch.empty(n, dtype=torch.float16, device=dev)
    mid = torch.empty(k, dtype=torch.float16, device=dev)
    b = torch.empty(m, dtype=torch.float16, device=dev)
    err = torch.empty(outer, dtype=torch.float32, device=dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    dbf_factorize(W.data_ptr(), n, m, k, U0.data_ptr(), V0.data_ptr(), d_out.data_ptr() if d_out is not None else 0,
                  d_in.data_ptr() if d_in is not None else 0, rho_rel, outer, inner, power_iters, A.data_ptr(),
                  B.data_ptr(), a.data_ptr(), mid.data_ptr(), b.data_ptr(), err.data_ptr(), stream)
    return A, B, a, mid, b, err


def dbf_linear_forward(h: int, x_ptr: int, y_ptr: int, batch: int, stream: int = 0) -> None:
    _check(lib().dbf_linear_forward(h, x_ptr, y_ptr, batch, stream), "dbf_linear_forward")


def dbf_linear_forward_ex(h: int, x_ptr: int, y_ptr: int, batch: int, path: int, stream: int = 0) -> None:
    _check(lib().dbf_linear_forward_ex(h, x_ptr, y_ptr, batch, path, stream), "dbf_linear_forward_ex")


def dbf_linear_forward_noalloc(h: int, x_ptr: int, y_ptr: int, batch: int, stream: int = 0) -> None:
    """dbf_linear_forward with the kernels' scratch in the library's static device array."""
    _check(lib().dbf_linear_forward_noalloc(h, x_ptr, y_ptr, batch, stream), "dbf_linear_forward_noalloc")


def dbf_linear_forward_group(hs, x_ptr: int, y_ptrs, batch: int, stream: int = 0) -> None:
    """Forwards of several layers that share the input x (device pointers)."""
    hs = list(hs)
    y_ptrs = list(y_ptrs)
    if len(hs) != len(y_ptrs):
        raise ValueError("one output per handle")
    harr = (ctypes.c_void_p * max(len(hs), 1))(*hs)
    yarr = (ctypes.c_void_p * max(len(y_ptrs), 1))(*y_ptrs)
    _check(lib().dbf_linear_forward_group(harr, len(hs), x_ptr, yarr, batch, stream), "dbf_linear_forward_group")


def forward_group(layers, x, outs=None, out_dtype=None):
    """ys[i] = layers[i](x) for Layer objects sharing the input width; one
    pair of launches for all of them at decode batch sizes.

    Where every layer is one of ``Layer.mx``, x may also be bfloat16 or an
    MxTensor, and the results float16 or bfloat16: out_dtype, by default the
    type of outs, without them x's (float16 for an MxTensor).
    """
    import torch
    if layers and all(L.act is not None for L in layers):
        return _forward_group_mx(layers, x, outs, out_dtype)
    if isinstance(x, MxTensor) or out_dtype not in (None, torch.float16) or x.dtype != torch.float16 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D float16 CUDA tensor")
    if any(L.m != x.shape[1] for L in layers):
        raise ValueError("x must have the layers' input width")
    if outs is None:
        outs = [torch.empty((x.shape[0], L.n), dtype=torch.float16, device=x.device) for L in layers]
    if len(outs) != len(layers):
        raise ValueError("one output per layer")
    for L, y in zip(layers, outs):
        if (y.dtype != torch.float16 or not y.is_cuda or tuple(y.shape) != (x.shape[0], L.n) or not y.is_contiguous()
                or y.device != x.device):
            raise ValueError("outs[i] must be a contiguous float16 tensor of shape (batch, n_i) on x's device")
    stream = torch.cuda.current_stream(x.device).cuda_stream
    dbf_linear_forward_group([L.handle for L in layers], x.data_ptr(), [y.data_ptr() for y in outs], x.shape[0],
                             stream)
    return outs


def _forward_group_mx(layers, x, outs, out_dtype):
    import torch
    m = layers[0].m
    if isinstance(x, MxTensor):
        like, scales, xt, default = x.codes, x.scales.data_ptr(), _TYPE_NAMES[x.fmt], torch.float16
        if x.cols != m:
            raise ValueError(f"x must have {m} columns")
    else:
        _check_rows(x, "x")
        like, scales, xt, default = x, None, _type_of(x.dtype), x.dtype
        if x.shape[1] != m:
            raise ValueError(f"x must have {m} columns")
    batch = like.shape[0]
    _check_count(batch, m)
    if out_dtype is None:
        out_dtype = outs[0].dtype if outs else default
    if out_dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("the outputs are float16 or bfloat16")
    if outs is None:
        outs = [like.new_empty((batch, L.n), dtype=out_dtype) for L in layers]
    if len(outs) != len(layers):
        raise ValueError("one output per layer")
    for L, y in zip(layers, outs):
        if (y.dtype != out_dtype or tuple(y.shape) != (batch, L.n) or not y.is_contiguous()
                or y.device != like.device):
            raise ValueError("outs[i] must be a contiguous tensor of shape (batch, n_i) of one type on x's device")
    n = len(layers)
    _call("dbf_mx_forward_group", like, (ctypes.c_void_p * n)(*[L.handle for L in layers]), n, like.data_ptr(), xt,
          scales, (ctypes.c_void_p * n)(*[y.data_ptr() for y in outs]), _type_of(out_dtype), batch)
    return outs


def norm_forward_group(layers, x, weight=None, residual=None, eps: float = 1e-6, outs=None):
    """(ys, norm) with norm = rms_norm(x, weight, residual, eps) and ys[i] = layers[i](norm.y): the norm in front of
    layers that share its result (gate and up, or q, k and v).

    Where every layer is one of ``Layer.mx`` that takes e4m3 blocks, the norm
    gives its rows in them and nothing is quantised again; otherwise they are
    in x's type (float16 for the other kinds of layers).  The results are in
    the type of outs, without them in x's.
    """
    import torch
    if x.dtype != torch.float16 and not all(L.act is not None for L in layers):
        raise ValueError("x must be float16 for layers that are not of Layer.mx")
    mx = all(L.act == "e4m3" for L in layers)
    norm = rms_norm(x, weight, residual, eps, mx=mx)
    return forward_group(layers, norm.y, outs, x.dtype if mx and not outs else None), norm


def dbf_linear_backward_data(h: int, dy_ptr: int, dx_ptr: int, batch: int, stream: int = 0) -> None:
    _check(lib().dbf_linear_backward_data(h, dy_ptr, dx_ptr, batch, stream), "dbf_linear_backward_data")


def dbf_linear_backward(h: int, x_ptr: int, dy_ptr: int, dx_ptr: int, da_ptr: int, dmid_ptr: int, db_ptr: int,
                        batch: int, stream: int = 0) -> None:
    _check(lib().dbf_linear_backward(h, x_ptr, dy_ptr, dx_ptr, da_ptr, dmid_ptr, db_ptr, batch, stream),
           "dbf_linear_backward")


def dbf_free(h: Optional[int]) -> None:
    lib().dbf_free(h)


def dbf_get_info(h: int) -> Dict[str, int]:
    info = _Info()
    _check(lib().dbf_get_info(h, ctypes.byref(info)), "dbf_get_info")
    return {name: getattr(info, name) for name, _ in _Info._fields_}


def dbf_pack_signs(S, words_per_row: Optional[int] = None) -> np.ndarray:
    """Pack a +/-1 matrix along its columns (host only)."""
    S = _as_signs(S)
    if S.ndim != 2:
        raise ValueError("S must be 2-D")
    rows, cols = S.shape
    wpr = (cols + 31) // 32 if words_per_row is None else int(words_per_row)
    out = np.zeros((rows, max(wpr, 1)), dtype=np.uint32)
    _check(lib().dbf_pack_signs(_ptr(S), rows, cols, _ptr(out), wpr), "dbf_pack_signs")
    return out


def dbf_layout_words(rows: int, words: int) -> int:
    return int(lib().dbf_layout_words(rows, words))


def dbf_layout_signs(packed: np.ndarray) -> np.ndarray:
    """Device tiling of packed signs (host only)."""
    packed = np.ascontiguousarray(packed, dtype=np.uint32)
    rows, words = packed.shape
    out = np.zeros(max(dbf_layout_words(rows, words), 1), dtype=np.uint32)
    _check(lib().dbf_layout_signs(_ptr(packed), rows, words, _ptr(out)), "dbf_layout_signs")
    return out


def dbf_layout_words_dec(rows_pad: int, cols_pad: int) -> int:
    return int(lib().dbf_layout_words_dec(rows_pad, cols_pad))


def dbf_layout_signs_dec(packed: np.ndarray, cols: int, rows_pad: int, cols_pad: int) -> np.ndarray:
    """The batch-1 decode kernels' copy of packed signs (host only)."""
    packed = np.ascontiguousarray(packed, dtype=np.uint32)
    rows, words = packed.shape
    out = np.zeros(max(dbf_layout_words_dec(rows_pad, cols_pad), 1), dtype=np.uint32)
    _check(lib().dbf_layout_signs_dec(_ptr(packed), rows, cols, words, rows_pad, cols_pad, _ptr(out)),
           "dbf_layout_signs_dec")
    return out


def dbf_timing_enable(h: int, enable: bool = True) -> None:
    _check(lib().dbf_timing_enable(h, 1 if enable else 0), "dbf_timing_enable")


def dbf_timing_read(h: int) -> Dict[str, Dict[str, float]]:
    """Per kernel name: launches and summed event time (ms) since the last read."""
    cap = 32
    buf = (_KernelTime * cap)()
    cnt = ctypes.c_int32()
    _check(lib().dbf_timing_read(h, buf, cap, ctypes.byref(cnt)), "dbf_timing_read")
    return {buf[i].name.decode(): {"launches": int(buf[i].launches), "total_ms": float(buf[i].total_ms)}
            for i in range(min(cnt.value, cap))}


_TYPE_NAMES = {"e4m3": DBF_TYPE_E4M3, "e2m1": DBF_TYPE_E2M1}


_TYPE_CODES: Dict[object, int] = {}


def _type_of(dtype) -> int:
    """The library's code of a torch dtype (-1: none)."""
    if not _TYPE_CODES:
        import torch
        _TYPE_CODES.update({torch.float16: DBF_TYPE_F16, torch.bfloat16: DBF_TYPE_BF16, torch.float32: DBF_TYPE_F32})
    return _TYPE_CODES.get(dtype, -1)


def _block_type(fmt: str) -> int:
    if fmt not in _TYPE_NAMES:
        raise ValueError("the block format is 'e4m3' or 'e2m1'")
    return _TYPE_NAMES[fmt]


def _call(where: str, t, *args) -> None:
    """lib().<where>(*args, stream) on t's device and its current stream.

    (The raw stream query takes 0.1 us of the host's time, a Stream object 1 to
    2; switching to the device that is current already another 1.)
    """
    import torch
    index = t.device.index
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _call(where, t, *args)
    status = getattr(_lib or lib(), where)(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != DBF_OK:
        raise DbfError(status, where)


class MxTensor:
    """A matrix in blocks of 32 columns with one power-of-two scale each (see
    "Block formats" in include/dbf.h).

    ``codes`` (uint8, rows x row bytes) and ``scales`` (uint8, rows x blocks)
    are contiguous CUDA tensors in the padded row layout; ``cols`` is the
    matrix's width and ``fmt`` is 'e4m3' (a byte per column) or 'e2m1' (half a
    byte).
    """

    __slots__ = ("codes", "scales", "cols", "fmt")

    def __init__(self, codes, scales, cols: int, fmt: str):
        import torch
        cols = int(cols)
        t = _block_type(fmt)
        if cols < 1:
            raise ValueError("cols must be positive")
        wide = -(-cols // 128) * 128
        row = wide if t == DBF_TYPE_E4M3 else wide // 2
        for a, width, what in ((codes, row, "codes"), (scales, wide // 32, "scales")):
            if a.dtype != torch.uint8 or not a.is_cuda or a.dim() != 2 or a.shape[1] != width or not a.is_contiguous():
                raise ValueError(f"{what} must be a contiguous CUDA uint8 tensor of shape (rows, {width})")
        if codes.shape[0] != scales.shape[0] or codes.device != scales.device:
            raise ValueError("codes and scales must have the same rows and device")
        self.codes, self.scales, self.cols, self.fmt = codes, scales, cols, fmt

    @property
    def shape(self):
        return (self.codes.shape[0], self.cols)

    @property
    def device(self):
        return self.codes.device

    def dequantize(self, dtype=None):
        """The values, as a tensor of `dtype` (float32, float16 or bfloat16; default float32)."""
        import torch
        dtype = torch.float32 if dtype is None else dtype
        t = _type_of(dtype)
        if t < 0:
            raise ValueError("dtype must be float32, float16 or bfloat16")
        out = self.codes.new_empty(self.shape, dtype=dtype)
        _call("dbf_mx_dequantize", out, self.codes.data_ptr(), self.scales.data_ptr(), _TYPE_NAMES[self.fmt],
              out.shape[0], self.cols, out.data_ptr(), t)
        return out


def _empty_blocks(rows: int, cols: int, fmt: str, like) -> MxTensor:
    """Uninitialised blocks on like's device."""
    import torch
    wide = -(-cols // 128) * 128
    q = MxTensor.__new__(MxTensor)  # (right by construction: __init__'s checks are for tensors of other origin)
    q.codes = like.new_empty((rows, wide if fmt == "e4m3" else wide // 2), dtype=torch.uint8)
    q.scales = like.new_empty((rows, wide // 32), dtype=torch.uint8)
    q.cols, q.fmt = cols, fmt
    return q


def mx_quantize(x, fmt: str = "e4m3") -> MxTensor:
    """x (contiguous 2-D CUDA tensor, float16, bfloat16 or float32) in blocks of 32 columns."""
    t = _type_of(x.dtype)
    ft = _block_type(fmt)
    if t < 0 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous() or x.shape[1] < 1:
        raise ValueError("x must be a contiguous 2-D CUDA tensor of float16, bfloat16 or float32")
    rows, cols = x.shape
    _check_count(rows, cols)
    q = _empty_blocks(rows, cols, fmt, x)
    _call("dbf_mx_quantize", x, x.data_ptr(), t, rows, cols, ft, q.codes.data_ptr(), q.scales.data_ptr())
    return q


def dbf_mx_pack(n: int, m: int, codes_ptr: int, scales_ptr: int, act_type: int, max_batch: int,
                stream: int = 0) -> int:
    """Handle of a layer with an e2m1 block weight (see dbf_mx_pack in include/dbf.h)."""
    h = ctypes.c_void_p()
    _check(lib().dbf_mx_pack(n, m, codes_ptr, scales_ptr, act_type, max_batch, stream, ctypes.byref(h)),
           "dbf_mx_pack")
    return h.value


def dbf_mx_forward_plan(batch: int, n: int, m: int, x_type: int):
    """(tile rows, tile columns, K parts) of a forward's product (see dbf_mx_forward_plan in include/dbf.h)."""
    plan = (ctypes.c_int32 * 3)()
    _check(lib().dbf_mx_forward_plan(batch, n, m, x_type, plan), "dbf_mx_forward_plan")
    return tuple(plan)


def dbf_mx_backward_plan(batch: int, n: int, m: int):
    """The same of an input gradient."""
    plan = (ctypes.c_int32 * 3)()
    _check(lib().dbf_mx_backward_plan(batch, n, m, plan), "dbf_mx_backward_plan")
    return tuple(plan)


class RmsNormOutput(NamedTuple):
    """y: the normalised rows (a tensor, or an e4m3 MxTensor); h: x + residual (x itself without a residual);
    rstd: 1 / rms of each row, float32."""
    y: object
    h: object
    rstd: object


def _check_count(rows: int, cols: int) -> None:
    if rows > 0x7fffffff or cols > 0x7fffffff:  # (the C ABI counts in int32)
        raise ValueError("more than 2^31 - 1 rows or columns")


def _check_rows(t, what, like=None):
    import torch
    if like is not None:  # (checked itself: its type, device and shape carry over)
        if t.dtype != like.dtype or t.shape != like.shape or t.device != like.device:
            raise ValueError(f"{what} must match the other rows in shape, type and device")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous 2-D CUDA tensor of float16 or bfloat16")
        return
    if t.dtype not in (torch.float16, torch.bfloat16) or not t.is_cuda or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 2-D CUDA tensor of float16 or bfloat16")
    _check_count(*t.shape)


def _check_norm_weight(weight, x) -> int:
    import torch
    if weight is None:
        return _type_of(x.dtype)
    if (weight.dtype not in (x.dtype, torch.float32) or tuple(weight.shape) != (x.shape[1],)
            or not weight.is_contiguous() or weight.device != x.device):
        raise ValueError("weight must be a contiguous vector of x's width and device, in x's type or float32")
    return _type_of(weight.dtype)


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6, mx: bool = False) -> RmsNormOutput:
    """Root-mean-square norm of the rows of x (+ residual): see dbf_rms_norm in include/dbf.h.

    x and residual are contiguous 2-D CUDA tensors (float16 or bfloat16).
    With ``mx`` the normalised rows come in e4m3 blocks, the input of
    ``Layer.mx`` layers; otherwise in x's type, the input of any layer.
    """
    import torch
    _check_rows(x, "x")
    if residual is not None:
        _check_rows(residual, "residual", x)
    wt = _check_norm_weight(weight, x)
    rows, cols = x.shape
    t = _type_of(x.dtype)
    h = torch.empty_like(x) if residual is not None else x
    rstd = x.new_empty(rows, dtype=torch.float32)
    if mx:
        y = _empty_blocks(rows, cols, "e4m3", x)
        y_ptr, s_ptr, yt = y.codes.data_ptr(), y.scales.data_ptr(), DBF_TYPE_E4M3
    else:
        y = torch.empty_like(x)
        y_ptr, s_ptr, yt = y.data_ptr(), None, t
    _call("dbf_rms_norm", x, x.data_ptr(), None if residual is None else residual.data_ptr(),
          None if weight is None else weight.data_ptr(), t, wt, rows, cols, eps,
          None if residual is None else h.data_ptr(), y_ptr, yt, s_ptr, rstd.data_ptr())
    return RmsNormOutput(y, h, rstd)


def rms_norm_backward(dy, h, weight, rstd, dh=None):
    """(dx, dweight) of rms_norm at its h and rstd: dx is the gradient of x and of the residual, with dh, the
    gradient that reaches h past the norm, added; dweight is float32 (also for weight=None)."""
    import torch
    _check_rows(dy, "dy")
    _check_rows(h, "h", dy)
    if dh is not None:
        _check_rows(dh, "dh", dy)
    wt = _check_norm_weight(weight, dy)
    rows, cols = dy.shape
    if rstd.dtype != torch.float32 or tuple(rstd.shape) != (rows,) or not rstd.is_contiguous() or rstd.device != dy.device:
        raise ValueError("rstd must be a contiguous float32 vector with one entry per row, on dy's device")
    dx = torch.empty_like(dy)
    dw = dy.new_empty(cols, dtype=torch.float32)
    nbytes = lib().dbf_rms_norm_backward_workspace(rows, cols)
    ws = dy.new_empty(max(nbytes, 16), dtype=torch.uint8)
    _call("dbf_rms_norm_backward", dy, dy.data_ptr(), h.data_ptr(), None if weight is None else weight.data_ptr(),
          rstd.data_ptr(), None if dh is None else dh.data_ptr(), _type_of(dy.dtype), wt, rows, cols, dx.data_ptr(),
          dw.data_ptr(), ws.data_ptr(), nbytes)
    return dx, dw


class RowGroups:
    """Rows in groups (see "Rows in groups" in include/dbf.h): ``order`` (int32, rows) holds the row at each place of
    the grouped order, ``offsets`` (int32, count + 1) the first place of each group and of the rows of no group.
    Contiguous CUDA vectors, as `group_rows` makes them."""

    __slots__ = ("order", "offsets")

    def __init__(self, order, offsets):
        import torch
        for a, what in ((order, "order"), (offsets, "offsets")):
            if a.dtype != torch.int32 or not a.is_cuda or a.dim() != 1 or not a.is_contiguous():
                raise ValueError(f"{what} must be a contiguous CUDA int32 vector")
        if offsets.numel() < 2 or order.device != offsets.device:
            raise ValueError("offsets must hold count + 1 entries, on order's device")
        self.order, self.offsets = order, offsets

    @property
    def rows(self) -> int:
        return self.order.numel()

    @property
    def count(self) -> int:
        return self.offsets.numel() - 1


def group_rows(index, count: int) -> RowGroups:
    """The grouped order of the rows that `index` (contiguous CUDA vector, int32 or int64) assigns to `count` groups;
    entries outside [0, count) are of no group.  Once for all the layers that the rows pass."""
    import torch
    if (index.dtype not in (torch.int32, torch.int64) or not index.is_cuda or index.dim() != 1
            or not index.is_contiguous()):
        raise ValueError("index must be a contiguous CUDA vector of int32 or int64")
    count, rows = int(count), index.numel()
    if not 1 <= count <= 1024 or rows > 1 << 24:
        raise ValueError("1 to 1024 groups and up to 2^24 rows")
    order = index.new_empty(rows, dtype=torch.int32)
    offsets = index.new_empty(count + 1, dtype=torch.int32)
    nbytes = lib().dbf_group_rows_workspace(rows, count)
    ws = index.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    _call("dbf_group_rows", index, index.data_ptr(), index.element_size() * 8, rows, count, order.data_ptr(),
          offsets.data_ptr(), None if ws is None else ws.data_ptr(), nbytes)
    g = RowGroups.__new__(RowGroups)  # (right by construction)
    g.order, g.offsets = order, offsets
    return g


def _check_groups(groups, count: int, rows: Optional[int], device) -> None:
    if not isinstance(groups, RowGroups):
        raise ValueError("groups must be the RowGroups of group_rows")
    if groups.count != count:
        raise ValueError(f"groups must have {count} groups")
    if rows is not None and groups.rows != rows:
        raise ValueError(f"groups must have {rows} rows")
    if groups.order.device != device:
        raise ValueError("groups must be on the rows' device")


def dbf_experts_pack(count: int, n: int, m: int, codes_ptr: int, scales_ptr: int, act_type: int, max_rows: int,
                     stream: int = 0) -> int:
    """Handle of experts with e2m1 block weights (see dbf_experts_pack in include/dbf.h)."""
    h = ctypes.c_void_p()
    _check(lib().dbf_experts_pack(count, n, m, codes_ptr, scales_ptr, act_type, max_rows, stream, ctypes.byref(h)),
           "dbf_experts_pack")
    return h.value


def dbf_experts_forward_plan(count: int, n: int, m: int, slots: int, x_type: int):
    """(tile rows, tile columns, most K parts, workgroups of a round, 1 for another launch before) of a product of
    experts (see dbf_experts_forward_plan in include/dbf.h)."""
    plan = (ctypes.c_int32 * 5)()
    _check(lib().dbf_experts_forward_plan(count, n, m, slots, x_type, plan), "dbf_experts_forward_plan")
    return tuple(plan)


def dbf_experts_backward_plan(count: int, n: int, m: int, slots: int):
    """The same of an input gradient."""
    plan = (ctypes.c_int32 * 5)()
    _check(lib().dbf_experts_backward_plan(count, n, m, slots, plan), "dbf_experts_backward_plan")
    return tuple(plan)


class Experts:
    """`count` 4-bit weights of n x m, each for the rows of one group (the experts of a sparse MLP).

    W is an e2m1 MxTensor of count * n rows, one weight after the other;
    max_rows is the most places (tokens times experts of a token) of a call.
    `groups` (of `group_rows`) assigns each place to an expert.  Calls on one
    object, forward and backward alike, share its workspace: on several
    streams they must be ordered, or each stream has an object of its own.
    """

    def __init__(self, W: MxTensor, count: int, max_rows: int, act: str = "e4m3"):
        import torch
        if not isinstance(W, MxTensor) or W.fmt != "e2m1":
            raise ValueError("W must be an e2m1 MxTensor")
        self.count = int(count)
        if self.count < 1 or W.shape[0] < 1 or W.shape[0] % self.count:
            raise ValueError("W must have the same number of rows for each of count weights")
        at = _block_type(act)
        self.n, self.m = W.shape[0] // self.count, W.cols
        self.max_rows, self.act = int(max_rows), act
        _check_count(self.n, self.max_rows)
        with torch.cuda.device(W.device):
            self.handle = dbf_experts_pack(self.count, self.n, self.m, W.codes.data_ptr(), W.scales.data_ptr(), at,
                                           self.max_rows, torch.cuda.current_stream().cuda_stream)

    def _rows(self, groups, gather: int, rows: int, device) -> int:
        """Checked number of places."""
        _check_groups(groups, self.count, None, device)
        slots = groups.rows
        if slots > self.max_rows:
            raise ValueError(f"more than {self.max_rows} rows")
        if gather < 0 or rows * max(gather, 1) != slots:
            raise ValueError("the rows must be one for each place, or with gather = k one for each k of them")
        return slots

    @staticmethod
    def _out(out, like, slots, width, dtype):
        if out is None:
            return like.new_empty((slots, width), dtype=dtype)
        if (tuple(out.shape) != (slots, width) or out.dtype != dtype or not out.is_contiguous()
                or out.device != like.device):
            raise ValueError(f"out must be a contiguous tensor of shape ({slots}, {width}) on the rows' device")
        return out

    def forward(self, x, groups: RowGroups, gather: int = 0, scatter: bool = False, out=None, out_dtype=None):
        """y[place] = x[row of the place] W_eᵀ, e the place's expert; zeros for places of none (see
        dbf_experts_forward in include/dbf.h).

        x: float16 or bfloat16 rows, quantised into `act` blocks by the call,
        or an MxTensor.  gather 0: x has a row for each place, in the grouped
        order; k: x is in the index's order, k consecutive entries share a
        row (tokens with k experts each).  scatter: results in the index's
        order instead of the grouped order.
        """
        import torch
        gather = int(gather)
        if isinstance(x, MxTensor):
            if x.cols != self.m:
                raise ValueError(f"x must have {self.m} columns")
            like, scales, xt, default = x.codes, x.scales.data_ptr(), _TYPE_NAMES[x.fmt], torch.float16
        else:
            _check_rows(x, "x")
            if x.shape[1] != self.m:
                raise ValueError(f"x must have {self.m} columns")
            like, scales, xt, default = x, None, _type_of(x.dtype), x.dtype
        slots = self._rows(groups, gather, like.shape[0], like.device)
        if out_dtype is None:
            out_dtype = default if out is None else out.dtype
        if out_dtype not in (torch.float16, torch.bfloat16):
            raise ValueError("the output is float16 or bfloat16")
        out = self._out(out, like, slots, self.n, out_dtype)
        _call("dbf_experts_forward", like, self.handle, like.data_ptr(), xt, scales, groups.order.data_ptr(),
              groups.offsets.data_ptr(), slots, gather, 1 if scatter else 0, out.data_ptr(), _type_of(out_dtype))
        return out

    __call__ = forward

    def backward_data(self, dy, groups: RowGroups, gather: int = 0, scatter: bool = False, out=None):
        """dx[place] = dy[row of the place] W_e for dy (float16 or bfloat16); gather and scatter as in forward."""
        gather = int(gather)
        _check_rows(dy, "dy")
        if dy.shape[1] != self.n:
            raise ValueError(f"dy must have {self.n} columns")
        slots = self._rows(groups, gather, dy.shape[0], dy.device)
        out = self._out(out, dy, slots, self.m, dy.dtype)
        _call("dbf_experts_backward_data", dy, self.handle, dy.data_ptr(), _type_of(dy.dtype),
              groups.order.data_ptr(), groups.offsets.data_ptr(), slots, gather, 1 if scatter else 0, out.data_ptr())
        return out

    def info(self) -> Dict[str, int]:
        return dbf_get_info(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            dbf_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class AdapterOutput(NamedTuple):
    """y: base + scale B A x; t: A x, float32 (rows x rank), which the backward pass takes."""
    y: object
    t: object


class Adapters:
    """`count` low-rank adapters beside a layer of any kind: y = base + scale_a B_a (A_a x) for rows of adapter a.

    A (count, rank, m) and B (count, n, rank) are contiguous CUDA tensors of
    float16 or bfloat16, scale a float32 vector or None (1).  They are read by
    each call and not copied, so a training step may change them in place.
    `groups` (of `group_rows`) assigns each row to an adapter, or to none.
    """

    def __init__(self, A, B, scale=None):
        import torch
        if A.dim() != 3 or B.dim() != 3 or A.shape[0] != B.shape[0] or A.shape[1] != B.shape[2] or 0 in A.shape + B.shape:
            raise ValueError("A must be (count, rank, m) and B (count, n, rank)")
        for a, what in ((A, "A"), (B, "B")):
            if (a.dtype not in (torch.float16, torch.bfloat16) or a.dtype != A.dtype or not a.is_cuda
                    or not a.is_contiguous() or a.device != A.device):
                raise ValueError(f"{what} must be a contiguous CUDA tensor of float16 or bfloat16, like A")
        if scale is not None and (scale.dtype != torch.float32 or tuple(scale.shape) != (A.shape[0],)
                                  or not scale.is_contiguous() or scale.device != A.device):
            raise ValueError("scale must be a contiguous float32 vector with one entry per adapter, on A's device")
        self.A, self.B, self.scale = A, B, scale
        self.count, self.rank, self.m = A.shape
        self.n = B.shape[1]
        self._sizes: Dict[tuple, int] = {}

    def _check(self, t, rows, width, what):
        if (t.dtype != self.A.dtype or t.dim() != 2 or t.shape != (rows, width) or not t.is_contiguous()
                or t.device != self.A.device):
            raise ValueError(f"{what} must be a contiguous tensor of shape ({rows}, {width}) in A's type on its device")

    def _workspace(self, of, rows):
        """Bytes that a call on so many rows needs (asked once for calls of the same size)."""
        known = self._sizes.get((of, rows))
        if known is None:
            if len(self._sizes) > 256:
                self._sizes.clear()
            known = self._sizes[of, rows] = getattr(lib(), of)(rows, self.n, self.m, self.rank, self.count)
        return known

    def _low(self, t, rows):
        import torch
        if t.dtype != torch.float32 or tuple(t.shape) != (rows, self.rank) or not t.is_contiguous() or t.device != self.A.device:
            raise ValueError(f"t must be a contiguous float32 tensor of shape ({rows}, {self.rank}) on A's device")

    def forward(self, x, base, groups: RowGroups, out=None) -> AdapterOutput:
        """(y, t) for rows x and the layer's results base; out may be base itself (see dbf_adapter_forward in
        include/dbf.h)."""
        import torch
        rows = x.shape[0] if x.dim() == 2 else 0
        self._check(x, rows, self.m, "x")
        self._check(base, rows, self.n, "base")
        _check_groups(groups, self.count, rows, x.device)
        if out is None:
            out = torch.empty_like(base)
        else:
            self._check(out, rows, self.n, "out")
        t = x.new_empty((rows, self.rank), dtype=torch.float32)
        nbytes = self._workspace("dbf_adapter_workspace", rows)
        ws = x.new_empty(max(nbytes, 16), dtype=torch.uint8)
        _call("dbf_adapter_forward", x, x.data_ptr(), base.data_ptr(), self.A.data_ptr(), self.B.data_ptr(),
              None if self.scale is None else self.scale.data_ptr(), _type_of(x.dtype), groups.order.data_ptr(),
              groups.offsets.data_ptr(), rows, self.n, self.m, self.rank, self.count, out.data_ptr(), t.data_ptr(),
              ws.data_ptr(), nbytes)
        return AdapterOutput(out, t)

    __call__ = forward

    def backward(self, dy, x, t, groups: RowGroups, dx=None, out=None):
        """(dx', dA, dB) at rows x with the forward's t for the upstream gradient dy: dx' = dx + scale (dy B) A with
        the layer's own input gradient dx (None: zeros); dA and dB are float32.  out (for dx') may be dx itself."""
        import torch
        rows = x.shape[0] if x.dim() == 2 else 0
        self._check(dy, rows, self.n, "dy")
        self._check(x, rows, self.m, "x")
        self._low(t, rows)
        _check_groups(groups, self.count, rows, x.device)
        for a, what in ((dx, "dx"), (out, "out")):
            if a is not None:
                self._check(a, rows, self.m, what)
        if out is None:
            out = torch.empty_like(x)
        elif out is x or out is dy:
            raise ValueError("out must not be x or dy")
        dA = x.new_empty(self.A.shape, dtype=torch.float32)
        dB = x.new_empty(self.B.shape, dtype=torch.float32)
        nbytes = self._workspace("dbf_adapter_backward_workspace", rows)
        ws = x.new_empty(max(nbytes, 16), dtype=torch.uint8)
        _call("dbf_adapter_backward", x, dy.data_ptr(), x.data_ptr(), t.data_ptr(),
              None if dx is None else dx.data_ptr(), self.A.data_ptr(), self.B.data_ptr(),
              None if self.scale is None else self.scale.data_ptr(), _type_of(x.dtype), groups.order.data_ptr(),
              groups.offsets.data_ptr(), rows, self.n, self.m, self.rank, self.count, out.data_ptr(), dA.data_ptr(),
              dB.data_ptr(), ws.data_ptr(), nbytes)
        return out, dA, dB


class Layer:
    """A DBF linear layer on the current GPU: ``y = layer(x)``.

    A (n x k) and B (k x m) are +/-1 arrays; a, mid, b are fp16 vectors.
    ``x`` is a contiguous fp16 CUDA (HIP) tensor of shape (batch, m) with
    batch <= max_batch; the result is a new fp16 tensor of shape (batch, n)
    computed on the current stream.
    """

    act: Optional[str] = None  # input blocks of a 4-bit layer (Layer.mx); None: a sign-factor layer

    def __init__(self, A, B, a, mid, b, max_batch: int = 2048, backward: bool = False):
        A = np.asarray(A)
        B = np.asarray(B)
        if A.ndim != 2 or B.ndim != 2 or A.shape[1] != B.shape[0]:
            raise ValueError("A must be n x k and B k x m")
        self.n, self.k = A.shape
        self.m = B.shape[1]
        self.max_batch = int(max_batch)
        self.handle = dbf_pack(self.n, self.m, self.k, A, B, a, mid, b, self.max_batch,
                               DBF_PACK_BACKWARD if backward else 0)

    @classmethod
    def bqq(cls, Y, Z, r, s, t, u, max_batch: int = 2048) -> "Layer":
        """A layer with the BQQ-form weight sum_i (r_i Y_i Z_i + s_i Y_i 1 + t_i 1 Z_i) + u 1:
        Y (p, n, d) and Z (p, d, m) of 0/1; forward only."""
        Y = np.asarray(Y)
        Z = np.asarray(Z)
        if Y.ndim != 3 or Z.ndim != 3 or Y.shape[0] != Z.shape[0] or Y.shape[2] != Z.shape[1]:
            raise ValueError("Y must be (p, n, d) and Z (p, d, m)")
        self = cls.__new__(cls)
        p, self.n, d = Y.shape
        self.m = Z.shape[2]
        self.k = p * d
        self.max_batch = int(max_batch)
        self.handle = dbf_bqq_pack(self.n, self.m, d, p, Y, Z, r, s, t, u, self.max_batch)
        return self

    @classmethod
    def bqq_grouped(cls, Y, Z, r, s, t, u, group: int, max_batch: int = 2048) -> "Layer":
        """A BQQ-form layer whose scalars r, s, t (p, ngroups) and u (ngroups,) change from one
        group of `group` input columns to the next; forward only."""
        Y = np.asarray(Y)
        Z = np.asarray(Z)
        if Y.ndim != 3 or Z.ndim != 3 or Y.shape[0] != Z.shape[0] or Y.shape[2] != Z.shape[1]:
            raise ValueError("Y must be (p, n, d) and Z (p, d, m)")
        self = cls.__new__(cls)
        p, self.n, d = Y.shape
        self.m = Z.shape[2]
        self.k = p * d
        self.max_batch = int(max_batch)
        self.handle = dbf_bqq_pack_grouped(self.n, self.m, d, p, int(group), Y, Z, r, s, t, u, self.max_batch)
        return self

    @classmethod
    def mx(cls, W: MxTensor, max_batch: int = 2048, act: str = "e4m3") -> "Layer":
        """A layer with a 4-bit weight W (n x m, an e2m1 MxTensor: `mx_quantize(w, "e2m1")`).

        Its forward takes float16 or bfloat16 rows, which are quantised into
        `act` blocks ('e4m3' or 'e2m1') by the call, or an MxTensor of either
        format; `backward_data` takes float16 or bfloat16.
        """
        if not isinstance(W, MxTensor) or W.fmt != "e2m1":
            raise ValueError("W must be an e2m1 MxTensor")
        at = _block_type(act)
        self = cls.__new__(cls)
        self.n, self.m = W.shape
        self.k = 0
        self.max_batch = int(max_batch)
        self.act = act
        import torch
        with torch.cuda.device(W.device):
            self.handle = dbf_mx_pack(self.n, self.m, W.codes.data_ptr(), W.scales.data_ptr(), at, self.max_batch,
                                      torch.cuda.current_stream().cuda_stream)
        return self

    def _forward_mx(self, x, out, path, out_dtype):
        import torch
        if path not in (DBF_PATH_AUTO, DBF_PATH_DECODE, DBF_PATH_PREFILL):
            raise DbfError(DBF_ERR_UNSUPPORTED, "Layer.forward")
        if isinstance(x, MxTensor):
            if x.cols != self.m:
                raise ValueError(f"x must have {self.m} columns")
            ptr, scales, xt, batch, default = x.codes.data_ptr(), x.scales.data_ptr(), _TYPE_NAMES[x.fmt], \
                x.codes.shape[0], torch.float16
        else:
            if (x.dtype not in (torch.float16, torch.bfloat16) or not x.is_cuda or x.dim() != 2
                    or x.shape[1] != self.m or not x.is_contiguous()):
                raise ValueError(f"x must be an MxTensor or a contiguous CUDA float16 or bfloat16 tensor of shape "
                                 f"(batch, {self.m})")
            ptr, scales, xt, batch, default = x.data_ptr(), None, _type_of(x.dtype), x.shape[0], x.dtype
        _check_count(batch, self.m)
        if path == DBF_PATH_DECODE and batch > DECODE_MAX_BATCH:
            raise DbfError(DBF_ERR_INVALID_ARG, "Layer.forward")
        if out is not None:
            default = out.dtype
        if out_dtype is None:
            out_dtype = default
        if out_dtype not in (torch.float16, torch.bfloat16):
            raise ValueError("the output is float16 or bfloat16")
        if out is None:
            out = (x.codes if isinstance(x, MxTensor) else x).new_empty((batch, self.n), dtype=out_dtype)
        elif (out.shape != (batch, self.n) or out.dtype != out_dtype or not out.is_contiguous()
              or out.device != x.device):
            raise ValueError("out must be a contiguous tensor of shape (batch, n) on x's device")
        _call("dbf_mx_forward", out, self.handle, ptr, xt, scales, out.data_ptr(), _type_of(out_dtype), batch)
        return out

    def info(self) -> Dict[str, int]:
        return dbf_get_info(self.handle)

    def forward(self, x, out=None, path: int = DBF_PATH_AUTO, out_dtype=None):
        import torch
        if self.act is not None:
            return self._forward_mx(x, out, path, out_dtype)
        if out_dtype not in (None, torch.float16):
            raise ValueError("the output is float16")
        if x.dtype != torch.float16 or not x.is_cuda or x.dim() != 2 or x.shape[1] != self.m:
            raise ValueError(f"x must be a CUDA float16 tensor of shape (batch, {self.m})")
        dev = getattr(self, "_device", None)
        if dev is None:
            dev = self._device = self.info()["device"]
        if x.device.index is not None and x.device.index != dev:
            raise ValueError("x must be on the layer's device")
        if not x.is_contiguous():
            raise ValueError("x must be contiguous")
        batch = x.shape[0]
        if out is None:
            out = torch.empty((batch, self.n), dtype=torch.float16, device=x.device)
        elif (out.shape != (batch, self.n) or out.dtype != torch.float16 or not out.is_contiguous()
              or not out.is_cuda or out.device != x.device):
            raise ValueError("out must be a contiguous float16 tensor of shape (batch, n) on x's device")
        stream = torch.cuda.current_stream(x.device).cuda_stream
        dbf_linear_forward_ex(self.handle, x.data_ptr(), out.data_ptr(), batch, path, stream)
        return out

    __call__ = forward

    @staticmethod
    def _check_act(t, width, what):
        import torch
        if t.dtype != torch.float16 or not t.is_cuda or t.dim() != 2 or t.shape[1] != width or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous CUDA float16 tensor of shape (batch, {width})")

    def backward_data(self, dy, out=None):
        """dX = dY W for dY of shape (batch, n); needs backward=True (Layer.mx: nothing, and dY may be bfloat16)."""
        import torch
        if self.act is not None:
            _check_rows(dy, "dy")
            if dy.shape[1] != self.n:
                raise ValueError(f"dy must have {self.n} columns")
            if out is None:
                out = dy.new_empty((dy.shape[0], self.m))
            elif (tuple(out.shape) != (dy.shape[0], self.m) or out.dtype != dy.dtype or not out.is_contiguous()
                  or out.device != dy.device):
                raise ValueError("out must be a contiguous tensor of shape (batch, m) in dy's type on its device")
            _call("dbf_mx_backward_data", dy, self.handle, dy.data_ptr(), out.data_ptr(), _type_of(dy.dtype),
                  dy.shape[0])
            return out
        self._check_act(dy, self.n, "dy")
        if out is None:
            out = torch.empty((dy.shape[0], self.m), dtype=torch.float16, device=dy.device)
        self._check_act(out, self.m, "out")
        if out.shape[0] != dy.shape[0] or out.device != dy.device:
            raise ValueError("out must have dy's batch and device")
        stream = torch.cuda.current_stream(dy.device).cuda_stream
        dbf_linear_backward_data(self.handle, dy.data_ptr(), out.data_ptr(), dy.shape[0], stream)
        return out

    def backward(self, x, dy):
        """(dX fp16, da, dmid, db fp32) at input x for upstream gradient dy; needs backward=True."""
        import torch
        self._check_act(x, self.m, "x")
        self._check_act(dy, self.n, "dy")
        if x.shape[0] != dy.shape[0] or x.device != dy.device:
            raise ValueError("x and dy must have the same batch and device")
        dev = x.device
        dx = torch.empty((x.shape[0], self.m), dtype=torch.float16, device=dev)
        da = torch.empty(self.n, dtype=torch.float32, device=dev)
        dmid = torch.empty(self.k, dtype=torch.float32, device=dev)
        db = torch.empty(self.m, dtype=torch.float32, device=dev)
        stream = torch.cuda.current_stream(dev).cuda_stream
        dbf_linear_backward(self.handle, x.data_ptr(), dy.data_ptr(), dx.data_ptr(), da.data_ptr(), dmid.data_ptr(),
                            db.data_ptr(), x.shape[0], stream)
        return dx, da, dmid, db

    def close(self) -> None:
        if getattr(self, "handle", None):
            dbf_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
