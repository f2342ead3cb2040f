"""ctypes binding of the C ABI in include/tiled_gemm.h.

Argument marshalling only: every step of the product runs in the CUDA
library.  The functions named like the C entry points take raw pointers
(ints), sizes and enum values and return the C status code.  `matmul` is the
convenience form for PyTorch CUDA tensors (PyTorch provides the device
memory and the stream); it raises GemmError on a non-zero status.

There is no fallback: if the library is missing or cannot be loaded, every
call raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading

from . import build as _build

F32, F16, BF16 = 0, 1, 2
DTYPE_CODES = {"f32": F32, "f16": F16, "bf16": BF16}

OK, ERR_INVALID_VALUE, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = 0, 1, 2, 3, 4

# The largest M, N or K the library accepts (GEMM_MAX_DIM).
MAX_DIM = (1 << 31) - 256

KERNELS = {
    "auto": 0,
    "simt": 1,
    "simt_tpb3": 2,
    "tc_128x128": 3,
    "tc_128x256": 4,
    "tc_256x256": 5,
    "tc_256x128": 6,
    "tc_small": 7,
    "tile16": 8,
}
KERNEL_NAMES = {v: k for k, v in KERNELS.items()}

HEADER = os.path.join(_build.ROOT, "include", "tiled_gemm.h")

_lock = threading.Lock()
_lib = None

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int

class Fp8Matrix(ctypes.Structure):
    """gemm_fp8_matrix_t: a quantised matrix in device memory."""

    _fields_ = [("data", _p), ("ld", _i64), ("type", _int), ("block", _int), ("scale", _p),
                ("scale_ld", _i64), ("op", _int)]


# The same layout as bytes, which are quicker to make.
_FP8_MATRIX = struct.Struct("@PqiiPqi4x")
assert _FP8_MATRIX.size == ctypes.sizeof(Fp8Matrix)
_pack_matrix = _FP8_MATRIX.pack


_SIGNATURES = {
    "gemm": ([_p, _p, _p, _i64, _i64, _i64, _int, _int, _p], _int),
    "gemm_ex": ([_p, _p, _p, _i64, _i64, _i64, _int, _int, _int, _p], _int),
    "gemm_ex_kernel": ([_p, _p, _p, _i64, _i64, _i64, _int, _int, _int, _int, _p], _int),
    "gemm_select_kernel": ([_p, _p, _p, _i64, _i64, _i64, _int, _int, _int], _int),
    "gemm_ws_split_count": ([_i64, _i64, _i64, _int, _int, _int], _int),
    "gemm_general": ([_p, _p, _p, _i64, _i64, _i64, _int, _int, ctypes.c_float, ctypes.c_float,
                      _int, _int, _int, _int, _p], _int),
    "gemm_ex_host": ([_p, _p, _p, _i64, _i64, _i64, _int, _int, _int, _p, _p, _p, _p], _int),
    "gemm_ex_host_ws": ([_p, _p, _p, _i64, _i64, _i64, _int, _int, _int, _p, _p, _p, _p,
                         ctypes.c_size_t, _p], _int),
    "gemm_host_panel_rows": ([_i64], _i64),
    "gemm_workspace_size": ([_i64, _i64, _i64], ctypes.c_size_t),
    "gemm_ex_ws": ([_p, _p, _p, _i64, _i64, _i64, _int, _int, _int, _p, ctypes.c_size_t, _p],
                   _int),
    "gemm_splitk_workspace_size": ([_i64, _i64, _i64, _int], ctypes.c_size_t),
    "gemm_splitk": ([_p, _p, _p, _i64, _i64, _i64, _int, _int, _int, _int, _p, ctypes.c_size_t,
                     _p], _int),
    "gemm_splitk_noalloc": ([_p, _p, _p, _i64, _i64, _i64, _int, _int, _int, _int, _p], _int),
    "gemm_fp8_quantize": ([_p, _i64, _i64, _i64, _int, _int, _int, _p, _i64, _p, _i64, _p], _int),
    "gemm_fp8_quantize_pair": ([_p, _i64, _i64, _i64, _int, _int, _p, _i64, _p, _i64, _p, _i64,
                                _p, _i64, _p], _int),
    "gemm_fp8": ([_p, _p, _p, _i64, _i64, _i64, _i64, ctypes.c_float, ctypes.c_float, _int, _p],
                 _int),
    "gemm_newton_schulz_workspace_size": ([_i64, _i64, _i64], ctypes.c_size_t),
    "gemm_newton_schulz": ([_p, _i64, _i64, _p, _i64, _i64, _i64, _i64, _i64, _int, _int, _int,
                            ctypes.POINTER(ctypes.c_float), ctypes.c_float, _p, ctypes.c_size_t,
                            _p], _int),
    "gemm_device_status": ([_p], _int),
    "gemm_debug_config": ([_i64, _int], _int),
    "gemm_launch_count": ([], ctypes.c_uint64),
    "gemm_traffic_model": ([_i64] * 9 + [_p], _int),
    "gemm_error_string": ([_int], ctypes.c_char_p),
}


class GemmError(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = code
        super().__init__(f"{where}: status {code} ({error_string(code)})")


def header_functions() -> list[str]:
    """Names of the functions declared in include/tiled_gemm.h."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)


def library_path() -> str:
    return _build.LIB_PATH


def load_library(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load the CUDA library (optionally building it first)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB_PATH
            if build_if_missing and not _build.up_to_date():
                _build.build()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"CUDA library {path} is not built; run "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            lib = ctypes.CDLL(path)
            for name, (args, res) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
    return _lib


def gemm(A, B, C, M, N, K, in_dtype, acc_dtype, stream=None) -> int:
    return load_library().gemm(A, B, C, M, N, K, in_dtype, acc_dtype, stream)


def gemm_ex(A, B, C, M, N, K, in_dtype, acc_dtype, out_dtype, stream=None) -> int:
    return load_library().gemm_ex(A, B, C, M, N, K, in_dtype, acc_dtype, out_dtype, stream)


def gemm_ex_kernel(A, B, C, M, N, K, in_dtype, acc_dtype, out_dtype, kernel, stream=None) -> int:
    return load_library().gemm_ex_kernel(A, B, C, M, N, K, in_dtype, acc_dtype, out_dtype,
                                         kernel, stream)


def gemm_general(A, B, C, M, N, K, op_a, op_b, alpha, beta, in_dtype, acc_dtype, out_dtype,
                 kernel=0, stream=None) -> int:
    return load_library().gemm_general(A, B, C, M, N, K, op_a, op_b, alpha, beta, in_dtype,
                                       acc_dtype, out_dtype, kernel, stream)


def gemm_select_kernel(A, B, C, M, N, K, in_dtype, acc_dtype, out_dtype) -> int:
    return load_library().gemm_select_kernel(A, B, C, M, N, K, in_dtype, acc_dtype, out_dtype)


def gemm_ex_host(A_host, B_host, C_host, M, N, K, in_dtype, acc_dtype, out_dtype, dA, dB, dC,
                 stream=None) -> int:
    return load_library().gemm_ex_host(A_host, B_host, C_host, M, N, K, in_dtype, acc_dtype,
                                       out_dtype, dA, dB, dC, stream)


def gemm_ex_host_ws(A_host, B_host, C_host, M, N, K, in_dtype, acc_dtype, out_dtype, dA, dB, dC,
                    workspace, workspace_bytes, stream=None) -> int:
    return load_library().gemm_ex_host_ws(A_host, B_host, C_host, M, N, K, in_dtype, acc_dtype,
                                          out_dtype, dA, dB, dC, workspace, workspace_bytes,
                                          stream)


def gemm_host_panel_rows(M) -> int:
    return load_library().gemm_host_panel_rows(M)


def gemm_workspace_size(M, N, K) -> int:
    return load_library().gemm_workspace_size(M, N, K)


def gemm_ws_split_count(M, N, K, in_dtype, acc_dtype, out_dtype) -> int:
    return load_library().gemm_ws_split_count(M, N, K, in_dtype, acc_dtype, out_dtype)


def gemm_ex_ws(A, B, C, M, N, K, in_dtype, acc_dtype, out_dtype, workspace, workspace_bytes,
               stream=None) -> int:
    return load_library().gemm_ex_ws(A, B, C, M, N, K, in_dtype, acc_dtype, out_dtype, workspace,
                                     workspace_bytes, stream)


def matmul_ws(A, B, out_dtype=None, workspace=None, out=None, stream=None):
    """C = A @ B through gemm_ex_ws (last-wave balancing with a workspace,
    allocated by PyTorch unless given)."""
    torch = _torch()
    M, K = A.shape
    N = B.shape[1]
    odt = torch.float32 if out_dtype is None else (
        torch_dtype(out_dtype) if isinstance(out_dtype, (str, int)) else out_dtype)
    C = out if out is not None else torch.empty((M, N), dtype=odt, device=A.device)
    if workspace is None:
        workspace = torch.empty(max(gemm_workspace_size(M, N, K), 16), dtype=torch.uint8,
                                device=A.device)
    nbytes = workspace.numel() * workspace.element_size()
    rc = gemm_ex_ws(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, dtype_code(A.dtype), F32,
                    dtype_code(C.dtype), workspace.data_ptr(), nbytes, _stream_handle(stream))
    if rc != OK:
        raise GemmError(rc, "gemm_ex_ws")
    return C


def gemm_splitk_workspace_size(M, N, K, splits) -> int:
    return load_library().gemm_splitk_workspace_size(M, N, K, splits)


def gemm_splitk(A, B, C, M, N, K, splits, in_dtype, acc_dtype, out_dtype, workspace,
                workspace_bytes, stream=None) -> int:
    return load_library().gemm_splitk(A, B, C, M, N, K, splits, in_dtype, acc_dtype, out_dtype,
                                      workspace, workspace_bytes, stream)


# Size of the library's fixed split-K scratch (GEMM_SPLITK_NOALLOC_MAX_BYTES).
SPLITK_NOALLOC_MAX_BYTES = 8 << 20


def gemm_splitk_noalloc(A, B, C, M, N, K, splits, in_dtype, acc_dtype, out_dtype,
                        stream=None) -> int:
    return load_library().gemm_splitk_noalloc(A, B, C, M, N, K, splits, in_dtype, acc_dtype,
                                              out_dtype, stream)


def matmul_splitk(A, B, splits: int, out_dtype=None, workspace=None, stream=None):
    """C = A @ B through gemm_splitk for contiguous CUDA tensors.  The FP32
    workspace is allocated by PyTorch unless given (a CUDA tensor of at
    least gemm_splitk_workspace_size bytes)."""
    torch = _torch()
    M, K = A.shape
    N = B.shape[1]
    odt = torch.float32 if out_dtype is None else (
        torch_dtype(out_dtype) if isinstance(out_dtype, (str, int)) else out_dtype)
    C = torch.empty((M, N), dtype=odt, device=A.device)
    need = gemm_splitk_workspace_size(M, N, K, splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=A.device)
    nbytes = workspace.numel() * workspace.element_size()
    rc = gemm_splitk(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, int(splits),
                     dtype_code(A.dtype), F32, dtype_code(odt), workspace.data_ptr(), nbytes,
                     _stream_handle(stream))
    if rc != OK:
        raise GemmError(rc, "gemm_splitk")
    return C


def gemm_fp8_quantize(X, ldx, rows, cols, in_dtype, f8, block, Q, ldq, S, lds,
                      stream=None) -> int:
    return load_library().gemm_fp8_quantize(X, ldx, rows, cols, in_dtype, f8, block, Q, ldq, S,
                                            lds, stream)


def gemm_fp8_quantize_pair(X, ldx, rows, cols, in_dtype, f8, Q_row, ldq_row, S_row, lds_row,
                           Q_col, ldq_col, S_col, lds_col, stream=None) -> int:
    return load_library().gemm_fp8_quantize_pair(X, ldx, rows, cols, in_dtype, f8, Q_row, ldq_row,
                                                 S_row, lds_row, Q_col, ldq_col, S_col, lds_col,
                                                 stream)


def gemm_fp8(A, B, C, ldc, M, N, K, alpha, beta, out_dtype, stream=None) -> int:
    """A and B: Fp8Matrix structures, or the bytes of such."""
    A, B = (ctypes.byref(m) if isinstance(m, Fp8Matrix) else m for m in (A, B))
    return load_library().gemm_fp8(A, B, C, ldc, M, N, K, alpha, beta, out_dtype, stream)


def gemm_newton_schulz_workspace_size(batch, rows, cols) -> int:
    return load_library().gemm_newton_schulz_workspace_size(batch, rows, cols)


def gemm_newton_schulz(G, ldg, batch_stride_g, O, ldo, batch_stride_o, batch, rows, cols, in_dtype,
                       out_dtype, steps, coefficients, eps, workspace, workspace_bytes,
                       stream=None) -> int:
    """coefficients: a ctypes array of 3 * steps floats (or None)."""
    return load_library().gemm_newton_schulz(G, ldg, batch_stride_g, O, ldo, batch_stride_o, batch,
                                             rows, cols, in_dtype, out_dtype, steps, coefficients,
                                             eps, workspace, workspace_bytes, stream)


def gemm_device_status(stream=None) -> int:
    return load_library().gemm_device_status(stream)


TRAFFIC_KEYS = ("a_elems", "b_elems", "c_elems", "bytes", "flops", "tiles", "steps",
                "ws_max", "ws_full")


def gemm_traffic_model(M, N, K, tm, tn, tk, in_bytes=2, acc_bytes=4, c_bytes=4) -> dict:
    """The library's closed-form traffic / working-set counts as a dict."""
    out = (ctypes.c_int64 * 9)()
    rc = load_library().gemm_traffic_model(M, N, K, tm, tn, tk, in_bytes, acc_bytes, c_bytes,
                                           out)
    if rc != OK:
        raise GemmError(rc, "gemm_traffic_model")
    return dict(zip(TRAFFIC_KEYS, list(out)))


def gemm_launch_count() -> int:
    return load_library().gemm_launch_count()


def gemm_debug_config(wait_budget_cycles: int = 0, fault_skip_kblock: int = -1) -> int:
    return load_library().gemm_debug_config(wait_budget_cycles, fault_skip_kblock)


def error_string(code: int) -> str:
    try:
        return load_library().gemm_error_string(code).decode()
    except RuntimeError:
        return "library not loaded"


gemm_error_string = error_string


# ------------------------------------------------------- PyTorch convenience

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_torch_dtype_codes = None


def _dtype_codes() -> dict:
    global _torch_dtype_codes
    if _torch_dtype_codes is None:
        torch = _torch()
        _torch_dtype_codes = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
    return _torch_dtype_codes


def dtype_code(dt) -> int:
    if isinstance(dt, str):
        return DTYPE_CODES[dt]
    return _dtype_codes()[dt]


def torch_dtype(code_or_name):
    torch = _torch()
    if isinstance(code_or_name, str):
        code_or_name = DTYPE_CODES[code_or_name]
    return {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}[code_or_name]


def _stream_handle(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


OPS = {"n": 0, "t": 1}


def addmm(A, B, C=None, op_a="n", op_b="n", alpha=1.0, beta=0.0, out_dtype=None,
          kernel: str | int = "auto", stream=None):
    """C = alpha * op(A) @ op(B) + beta * C for contiguous CUDA tensors, in place
    in C when given (C is allocated, and beta must be 0, otherwise).

    op "n" takes an operand as stored, "t" its transpose (A stored K x M, B
    stored N x K).  Returns C without synchronizing."""
    torch = _torch()
    if A.dim() != 2 or B.dim() != 2 or A.dtype != B.dtype:
        raise ValueError("A and B must be 2-D tensors of one dtype")
    if not (A.is_cuda and B.is_cuda and A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous CUDA tensors")
    ta, tb = OPS[op_a], OPS[op_b]
    M, K = (A.shape[1], A.shape[0]) if ta else (A.shape[0], A.shape[1])
    K2, N = (B.shape[1], B.shape[0]) if tb else (B.shape[0], B.shape[1])
    if K != K2:
        raise ValueError("inner dimensions differ")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        odt = torch.float32 if out_dtype is None else torch_dtype(out_dtype) \
            if isinstance(out_dtype, (str, int)) else out_dtype
        C = torch.empty((M, N), dtype=odt, device=A.device)
    elif tuple(C.shape) != (M, N) or not C.is_contiguous() or not C.is_cuda:
        raise ValueError("C must be a contiguous (M, N) CUDA tensor")
    kid = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    rc = gemm_general(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, ta, tb, float(alpha),
                      float(beta), dtype_code(A.dtype), F32, dtype_code(C.dtype), kid,
                      _stream_handle(stream))
    if rc != OK:
        raise GemmError(rc, "gemm_general")
    return C


def matmul(A, B, out_dtype=None, kernel: str | int = "auto", out=None, stream=None):
    """C = A @ B for contiguous row-major CUDA tensors (FP32 accumulation).

    out_dtype defaults to FP32 (the accumulator type); `out` may supply a
    preallocated contiguous (M, N) tensor of that type.  Runs on `stream`
    (default: PyTorch's current stream) and returns without synchronizing.
    """
    torch = _torch()
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"bad shapes {tuple(A.shape)} @ {tuple(B.shape)}")
    if A.dtype != B.dtype:
        raise TypeError("A and B must have the same dtype")
    if not (A.is_cuda and B.is_cuda):
        raise ValueError("A and B must be CUDA tensors")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous row-major")
    M, K = A.shape
    N = B.shape[1]
    odt = torch.float32 if out_dtype is None else (
        torch_dtype(out_dtype) if isinstance(out_dtype, (str, int)) else out_dtype)
    if out is None:
        out = torch.empty((M, N), dtype=odt, device=A.device)
    elif out.shape != (M, N) or out.dtype != odt or not out.is_contiguous():
        raise ValueError("out must be a contiguous (M, N) tensor of the output dtype")
    kid = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    rc = gemm_ex_kernel(A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N, K,
                        dtype_code(A.dtype), F32, dtype_code(odt), kid, _stream_handle(stream))
    if rc != OK:
        raise GemmError(rc, "gemm_ex_kernel")
    return out


# ------------------------------------------------- block-scaled 8-bit products

E4M3, E5M2 = 0, 1
F8_CODES = {"e4m3": E4M3, "e5m2": E5M2}
FP8_BLOCKS = {"row": 0, "col": 1, "tile": 2}


def _empty(shape, dtype, device):
    return (_cached or _cache()).empty(shape, dtype=dtype, device=device)


def _out_dtype(out_dtype):
    torch = _torch()
    if out_dtype is None:
        return torch.float32
    return torch_dtype(out_dtype) if isinstance(out_dtype, (str, int)) else out_dtype


def _f8_code(dtype) -> int:
    if isinstance(dtype, str):
        if dtype not in F8_CODES:
            raise ValueError(f"unknown 8-bit type {dtype!r}")
        return F8_CODES[dtype]
    code = _cache().f8_codes.get(dtype)
    if code is None:
        raise TypeError(f"{dtype} is not an 8-bit floating-point type")
    return code


class _Torch:
    """What the calls below take from PyTorch, looked up once: they spend
    about 10 us of host time in all, so that every look-up shows."""

    def __init__(self):
        torch = _torch()
        self.current_device = torch._C._cuda_getDevice
        # the address of the current stream, 3 us less than building a Stream object
        self.current_stream = torch._C._cuda_getCurrentRawStream
        self.empty = torch.empty
        self.float32 = torch.float32
        self.f8_types = (torch.float8_e4m3fn, torch.float8_e5m2)
        self.f8_codes = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}
        self.codes = _dtype_codes()


_cached = None


def _cache() -> _Torch:
    global _cached
    if _cached is None:
        _cached = _Torch()
    return _cached


def _allocate(stream, make, *args):
    """make(*args) with PyTorch allocating for `stream` (memory freed later is
    then reused in that stream's order only)."""
    if stream is None:
        return make(*args)
    with _torch().cuda.stream(stream):
        return make(*args)


def _stream_ptr(stream, x) -> int:
    """The stream's address; by default the current one of x's device."""
    if stream is not None:
        return stream.cuda_stream
    return (_cached or _cache()).current_stream(x.get_device())


def _check_matrix(x, what):
    """Returns (rows, cols, row stride) of a 2-D tensor with contiguous rows on
    the current CUDA device."""
    device = x.get_device()
    shape = x.shape
    if device < 0 or len(shape) != 2:
        raise ValueError(f"{what} must be a 2-D CUDA tensor")
    if device != (_cached or _cache()).current_device():
        raise ValueError(f"{what} is not on the current device")
    rows, cols = shape
    pitch, step = x.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what}'s rows must be contiguous")
    if rows <= 1:  # a single row has no pitch of its own
        return rows, cols, (cols + 15) // 16 * 16
    if pitch < cols:
        raise ValueError(f"{what}'s rows must not overlap")
    return rows, cols, pitch


def _fp8_empty(rows, cols, f8, block, device):
    """Uninitialised codes with a row pitch of a multiple of 16, their pitch,
    scales and their pitch."""
    t = _cached or _cache()
    ld = (cols + 15) // 16 * 16
    q = t.empty((rows, ld), device=device, dtype=t.f8_types[f8])
    if ld != cols:
        q = q[:, :cols]
    if block == 0:
        n, lds = (cols + 127) // 128, rows
    else:
        n, lds = (rows + 127) // 128, cols if block == 1 else (cols + 127) // 128
    return q, ld, t.empty((n, lds), device=device, dtype=t.float32), lds


def _quantize_input(x):
    """(rows, cols, row stride, type code) of a tensor to quantise."""
    rows, cols, ldx = _check_matrix(x, "x")
    code = (_cached or _cache()).codes.get(x.dtype)
    if code is None:
        raise TypeError("x must be FP32, FP16 or BF16")
    return rows, cols, ldx, code


def quantize_fp8(x, block: str = "row", dtype="e4m3", stream=None):
    """Quantise a 2-D CUDA tensor (FP32, FP16 or BF16; rows contiguous, any
    row stride) into 8-bit floating point with one FP32 scale for each block
    of 128.

    block: "row" (1 x 128; scales of shape (ceil(cols / 128), rows)), "col"
    (128 x 1; (ceil(rows / 128), cols)) or "tile" (128 x 128;
    (ceil(rows / 128), ceil(cols / 128))).  dtype: "e4m3" or "e5m2".  Returns
    (codes, scales): an element is its code times its block's scale.  The
    codes are a (rows, cols) view of rows padded to 16 bytes, the form
    matmul_fp8 takes.  The scales' attribute `fp8_block` says the block shape.
    The exact definition is gemm_fp8_quantize's.
    """
    rows, cols, ldx, code = _quantize_input(x)
    kind = FP8_BLOCKS.get(block)
    if kind is None:
        raise ValueError(f"unknown block shape {block!r}")
    f8 = _f8_code(dtype)
    q, ldq, s, lds = _allocate(stream, _fp8_empty, rows, cols, f8, kind, x.device)
    rc = (_lib or load_library()).gemm_fp8_quantize(
        x.data_ptr(), ldx, rows, cols, code, f8, kind, q.data_ptr(), ldq, s.data_ptr(), lds,
        _stream_ptr(stream, x))
    if rc != OK:
        raise GemmError(rc, "gemm_fp8_quantize")
    s.fp8_block = block
    return q, s


def quantize_fp8_pair(x, dtype="e4m3", stream=None):
    """quantize_fp8 with "row" and with "col" blocks from one read of x:
    ((codes, scales), (codes, scales))."""
    rows, cols, ldx, code = _quantize_input(x)
    f8 = _f8_code(dtype)
    qr, ldr, sr, ldsr = _allocate(stream, _fp8_empty, rows, cols, f8, 0, x.device)
    qc, ldc, sc, ldsc = _allocate(stream, _fp8_empty, rows, cols, f8, 1, x.device)
    rc = (_lib or load_library()).gemm_fp8_quantize_pair(
        x.data_ptr(), ldx, rows, cols, code, f8, qr.data_ptr(), ldr, sr.data_ptr(), ldsr,
        qc.data_ptr(), ldc, sc.data_ptr(), ldsc, _stream_ptr(stream, x))
    if rc != OK:
        raise GemmError(rc, "gemm_fp8_quantize_pair")
    sr.fp8_block, sc.fp8_block = "row", "col"
    return (qr, sr), (qc, sc)


def _fp8_operand(q, s, op, k_rows, kind, what):
    """(stored rows, stored columns, the bytes of its gemm_fp8_matrix_t) of
    codes q and scales s; k_rows: q's rows run along K.  kind: the scales'
    block shape, where the caller says it."""
    rows, cols, ld = _check_matrix(q, what)
    t = _cached or _cache()
    if s.dtype is not t.float32 or s.dim() != 2 or not s.is_contiguous() \
            or s.get_device() != q.get_device():
        raise ValueError(f"{what}'s scales must be a contiguous 2-D FP32 tensor on its device")
    rb, cb = (rows + 127) // 128, (cols + 127) // 128
    n, lds = s.shape
    if kind is not None and kind not in FP8_BLOCKS:
        raise ValueError(f"unknown block shape {kind!r}")
    if k_rows and n == cb and lds == rows:
        block = 0
    elif not k_rows and n == rb and lds == cols:
        block = 1
    elif n == rb and lds == cb:
        block = 2
    else:
        raise ValueError(f"{what}'s scales have shape {(n, lds)}: expected "
                         f"{(cb, rows) if k_rows else (rb, cols)} (a vector along the "
                         f"contraction) or {(rb, cb)} (128 x 128 blocks)")
    # A square matrix's two vector shapes have scales of the same shape: what
    # quantised it (or the caller) says which one it is.  (Of one element, all
    # shapes are the same.)
    if rows == cols and rows > 1:
        kind = kind or getattr(s, "fp8_block", None)
        if FP8_BLOCKS.get(kind, block) != block:
            raise ValueError(f"{what} has {kind!r} blocks: a scale vector must run along the "
                             "contraction")
    f8 = t.f8_codes.get(q.dtype)
    if f8 is None:
        raise TypeError(f"{what} must have an 8-bit floating-point type")
    return rows, cols, _pack_matrix(q.data_ptr(), ld, f8, block, s.data_ptr(), lds, op)


def matmul_fp8(a, a_scale, b, b_scale, op_a="n", op_b="t", out_dtype=None, out=None, alpha=1.0,
               beta=0.0, stream=None, block_a=None, block_b=None):
    """C = alpha * op(A) @ op(B) + beta * C on quantised operands, as
    quantize_fp8 gives them (FP32 accumulation; the scales are applied for
    each 128 of the contraction).

    op "n" takes an operand as stored, "t" its transpose; the defaults are
    x @ W^T with W stored out x in.  A scale vector must run along the
    contraction: "row" blocks where the stored rows do, "col" blocks
    otherwise; "tile" blocks serve both.  The scales' shape tells the block
    shape, but for a square matrix's two vectors: those are told apart by
    block_a and block_b ("row", "col" or "tile"), else by the `fp8_block`
    that quantize_fp8 sets on its scales, and are taken to run along the
    contraction where neither is there.  `out` may supply C (rows
    contiguous, any row stride); beta != 0 needs it.  out_dtype defaults to
    FP32, or to out's type.  Returns C without synchronizing."""
    ta, tb = OPS.get(op_a), OPS.get(op_b)
    if ta is None or tb is None:
        raise ValueError("op_a and op_b are \"n\" or \"t\"")
    M, K, A = _fp8_operand(a, a_scale, ta, not ta, block_a, "a")
    K2, N, B = _fp8_operand(b, b_scale, tb, tb, block_b, "b")
    if ta:
        M, K = K, M
    if tb:
        K2, N = N, K2
    if K != K2:
        raise ValueError("inner dimensions differ")
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs out")
        out = _allocate(stream, _empty, (M, N), _out_dtype(out_dtype), a.device)
        ldc = N
    else:
        rows, cols, ldc = _check_matrix(out, "out")
        if (rows, cols) != (M, N) or (out_dtype is not None and
                                      out.dtype != _out_dtype(out_dtype)):
            raise ValueError("out must be an (M, N) tensor of the output dtype")
    rc = (_lib or load_library()).gemm_fp8(A, B, out.data_ptr(), ldc, M, N, K, alpha, beta,
                                           dtype_code(out.dtype), _stream_ptr(stream, a))
    if rc != OK:
        raise GemmError(rc, "gemm_fp8")
    return out


# ------------------------------------------------------------ orthogonalisation

# Coefficients of one step that bring singular values from about 0.01 into
# [0.7, 1.2] in five steps.
NEWTON_SCHULZ_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def newton_schulz(G, steps: int = 5, coefficients=NEWTON_SCHULZ_COEFFICIENTS, eps: float = 1e-7,
                  out_dtype=None, out=None, workspace=None, stream=None):
    """Orthogonalise a CUDA matrix (or a batch of them, 3-D) by Newton-Schulz
    products, as the Muon optimiser does with a gradient's running mean:
    X = G / (norm + eps), then `steps` times A = X X^T, X = a X + (b A + c A A) X.

    G: FP32, FP16 or BF16, rows contiguous, any row and batch stride that
    keeps the matrices apart (also row by row, as t.transpose(0, 1) does), or
    one matrix expanded over the batch.
    coefficients: one (a, b, c) for every step, or a sequence of `steps` of
    them.  out_dtype defaults to G's type; `out` may supply the result (it
    may be G itself).  workspace: a CUDA tensor of at least
    gemm_newton_schulz_workspace_size(batch, rows, cols) bytes, allocated by
    PyTorch unless given.  Accuracy goes by the result's type: BF16 results are
    within 2e-3 of exact arithmetic before they are rounded (1.7e-3), FP32 and
    FP16 ones (and all with a side of up to 128) within about 1e-5, for up to
    three times the time, for five steps of the default coefficients; see
    gemm_newton_schulz in the header.
    Returns the result without synchronizing."""
    batch, rows, cols, ldg, stride_g = _check_batch(G, "G")
    if not 1 <= steps <= 32:
        raise ValueError("steps must be between 1 and 32")
    if len(coefficients) == 3 and not hasattr(coefficients[0], "__len__"):
        values = (*coefficients,) * steps
    else:
        if len(coefficients) != steps or any(len(r) != 3 for r in coefficients):
            raise ValueError("coefficients are (a, b, c), or one such triple for each step")
        values = [v for r in coefficients for v in r]
    if out is None:
        odt = G.dtype if out_dtype is None else _out_dtype(out_dtype)
        out = _allocate(stream, _empty, G.shape, odt, G.device)
        ldo, stride_o = cols, rows * cols
    else:
        *_, ldo, stride_o = _check_batch(out, "out")
        if out.shape != G.shape or (out_dtype is not None and out.dtype != _out_dtype(out_dtype)):
            raise ValueError("out must have G's shape and the output dtype")
    lib = _lib or load_library()
    if workspace is None:
        nbytes = lib.gemm_newton_schulz_workspace_size(batch, rows, cols)
        workspace = _allocate(stream, _empty, (nbytes,), _torch().uint8, G.device)
    elif workspace.get_device() != G.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on G's device")
    else:
        nbytes = workspace.numel() * workspace.element_size()
    rc = lib.gemm_newton_schulz(G.data_ptr(), ldg, stride_g, out.data_ptr(), ldo, stride_o, batch,
                                rows, cols, dtype_code(G.dtype), dtype_code(out.dtype), steps,
                                (ctypes.c_float * (3 * steps))(*values), eps,
                                workspace.data_ptr(), nbytes, _stream_ptr(stream, G))
    if rc != OK:
        raise GemmError(rc, "gemm_newton_schulz")
    return out


def _check_batch(x, what):
    """(batch, rows, cols, row stride, batch stride) of a matrix or a 3-D batch."""
    if x.dim() not in (2, 3) or not x.is_cuda:
        raise ValueError(f"{what} must be a 2-D or 3-D CUDA tensor")
    if x.dtype not in (_cached or _cache()).codes:
        raise TypeError(f"{what} must be FP32, FP16 or BF16")
    if x.dim() == 2:
        return 1, *_check_matrix(x, what), 0
    if x.shape[0] == 0:
        return 0, x.shape[1], x.shape[2], x.shape[2], 0
    return x.shape[0], *_check_matrix(x[0], what), x.stride(0)
