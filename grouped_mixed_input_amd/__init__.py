"""grouped_mixed_input_amd -- grouped, mixed-input (W4A16) and implicit-conv GEMM
for AMD MI355X (gfx950).

A thin binding over the C ABI of ``libgmi.so`` (declared in
``include/gmi.h``): ctypes, and for the calls whose device time is a few
microseconds the native module ``_calls``.  Functions here only marshal torch
tensors into device pointers, sizes and the current HIP stream; every step of
the computation runs in the library's HIP kernels.  There is no fallback: if ``libgmi.so`` has not
been built, importing the binding's functions raises.
"""
from __future__ import annotations

import ctypes
import pathlib
from typing import NamedTuple

import torch

_PKG = pathlib.Path(__file__).resolve().parent
LIB_PATH = _PKG / "libgmi.so"

GMI_OK, GMI_ERR_INVALID_ARG, GMI_ERR_UNSUPPORTED, GMI_ERR_MISALIGNED, GMI_ERR_WORKSPACE, GMI_ERR_HIP = range(6)
STATUS_NAMES = ["GMI_OK", "GMI_ERR_INVALID_ARG", "GMI_ERR_UNSUPPORTED", "GMI_ERR_MISALIGNED", "GMI_ERR_WORKSPACE",
                "GMI_ERR_HIP"]
GMI_F16, GMI_BF16, GMI_F8E4M3, GMI_F32 = 0, 1, 2, 3
_DT = {torch.float16: GMI_F16, torch.bfloat16: GMI_BF16, torch.float8_e4m3fn: GMI_F8E4M3}


class GmiError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"{name}: {message}")


class Problem(ctypes.Structure):
    """Mirror of gmi_problem."""
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldc", ctypes.c_int64), ("ldd", ctypes.c_int64),
                ("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("C", ctypes.c_void_p), ("D", ctypes.c_void_p)]


_lib = None
_i32, _i64, _f32, _p, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """Load libgmi.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not LIB_PATH.exists():
        raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                           "python -m grouped_mixed_input_amd.build")
    L = ctypes.CDLL(str(LIB_PATH))
    L.gmi_last_error.restype = ctypes.c_char_p
    L.gmi_last_error.argtypes = []
    L.gmi_workspace_bytes.restype = _sz
    L.gmi_workspace_bytes.argtypes = [_i32]
    L.gmi_gemm_grouped.restype = ctypes.c_int
    L.gmi_gemm_grouped.argtypes = [ctypes.POINTER(Problem), _i32, ctypes.c_int, _f32, _f32, _p, _sz, _p]
    L.gmi_gemm_grouped_offsets.restype = ctypes.c_int
    L.gmi_gemm_grouped_offsets.argtypes = [_i32, _p, _i32, _i32, _i32, _p, _i64, _p, _i64, _i64, _p, _i64, _p, _i64,
                                           ctypes.c_int, _f32, _f32, _p, _sz, _p]
    L.gmi_gemm_grouped_offsets_noalloc.restype = ctypes.c_int
    L.gmi_gemm_grouped_offsets_noalloc.argtypes = [_i32, _p, _i32, _i32, _i32, _p, _i64, _p, _i64, _i64, _p, _i64, _p,
                                                   _i64, ctypes.c_int, _f32, _f32, _p]
    L.gmi_gemm_ptr_array.restype = ctypes.c_int
    L.gmi_gemm_ptr_array.argtypes = [_i32, _i32, _i32, _i32, _p, _i64, _p, _i64, _p, _i64, _p, _i64, ctypes.c_int,
                                     _f32, _f32, _p]
    L.gmi_prepack_w4_bytes.restype = _sz
    L.gmi_prepack_w4_bytes.argtypes = [_i32, _i32]
    L.gmi_prepack_w4.restype = ctypes.c_int
    L.gmi_prepack_w4.argtypes = [_p, _i32, _i32, _p, _p]
    L.gmi_gemm_w4a16.restype = ctypes.c_int
    L.gmi_gemm_w4a16.argtypes = [_i32, _i32, _i32, _p, _i64, _p, _p, _p, _i32, _p, _i64, _p, _sz, _p]
    L.gmi_gemm_mixed.restype = ctypes.c_int
    L.gmi_gemm_mixed.argtypes = [_i32, _i32, _i32, ctypes.c_int, _p, _i64, _p, ctypes.c_int, _p, _p, _i32, _p, _i64,
                                 _p, _sz, _p]
    L.gmi_gemm_mixed_grouped.restype = ctypes.c_int
    L.gmi_gemm_mixed_grouped.argtypes = [_i32, _p, _i32, _i32, _i32, ctypes.c_int, _p, _i64, _p, _i64, ctypes.c_int,
                                         _p, _i64, _p, _i64, _i32, _p, _i64, _p]
    L.gmi_conv2d_fprop_implicit_fused.restype = ctypes.c_int
    L.gmi_conv2d_fprop_implicit_fused.argtypes = [_i32] * 13 + [_p, _p, _p, _p, _p, ctypes.c_int, _f32, _f32,
                                                               ctypes.c_int, _p]
    L.gmi_conv2d_dgrad_workspace_bytes.restype = _sz
    L.gmi_conv2d_dgrad_workspace_bytes.argtypes = [_i32] * 4
    L.gmi_conv2d_dgrad_implicit.restype = ctypes.c_int
    L.gmi_conv2d_dgrad_implicit.argtypes = [_i32] * 13 + [_p, _p, _p, _p, ctypes.c_int, _f32, _f32, _p, _sz, _p]
    L.gmi_conv2d_wgrad_workspace_bytes.restype = _sz
    L.gmi_conv2d_wgrad_workspace_bytes.argtypes = [_i32] * 14
    L.gmi_conv2d_wgrad_implicit.restype = ctypes.c_int
    L.gmi_conv2d_wgrad_implicit.argtypes = [_i32] * 14 + [_p, _p, _p, _p, ctypes.c_int, _f32, _f32, _p, _sz, _p]
    L.gmi_w4a16_workspace_bytes.restype = _sz
    L.gmi_w4a16_workspace_bytes.argtypes = [_i32, _i32, _i32]
    L.gmi_conv2d_fprop_implicit.restype = ctypes.c_int
    L.gmi_conv2d_fprop_implicit.argtypes = [_i32] * 13 + [_p, _p, _p, _p, ctypes.c_int, _f32, _f32, _p]
    L.gmi_time_next_gemm.restype = ctypes.c_int
    L.gmi_time_next_gemm.argtypes = [_p, _p]
    L.gmi_rmsnorm_quant.restype = ctypes.c_int
    L.gmi_rmsnorm_quant.argtypes = [_i32, _i32, _p, _i64, _p, _i64, _p, _f32, ctypes.c_int, _p, _i64, _p, _i64, _p,
                                    _i64, _p, _i64, _p]
    L.gmi_rmsnorm_bwd_workspace_bytes.restype = _sz
    L.gmi_rmsnorm_bwd_workspace_bytes.argtypes = [_i32, _i32]
    L.gmi_rmsnorm_bwd.restype = ctypes.c_int
    L.gmi_rmsnorm_bwd.argtypes = [_i32, _i32, _p, _i64, _p, _i64, _p, _p, _i64, _f32, ctypes.c_int, _p, _i64, _p, _p,
                                  _sz, _p]
    L.gmi_gemm_f8_block_workspace_bytes.restype = _sz
    L.gmi_gemm_f8_block_workspace_bytes.argtypes = [_i32] * 3
    L.gmi_gemm_f8_block.restype = ctypes.c_int
    L.gmi_gemm_f8_block.argtypes = [_i32, _i32, _i32, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _sz, _p]
    L.gmi_gemm_f8_block_grouped_workspace_bytes.restype = _sz
    L.gmi_gemm_f8_block_grouped_workspace_bytes.argtypes = [_i32]
    L.gmi_gemm_f8_block_grouped.restype = ctypes.c_int
    L.gmi_gemm_f8_block_grouped.argtypes = [_i32, _p, _i32, _i32, _i32, _p, _i64, _p, _i64, _p, _i64, _i64, _p, _i64,
                                            _i64, _p, _i64, _p, _sz, _p]
    L.gmi_moe_route_workspace_bytes.restype = _sz
    L.gmi_moe_route_workspace_bytes.argtypes = [_i32, _i32]
    L.gmi_moe_route.restype = ctypes.c_int
    L.gmi_moe_route.argtypes = [_i32, _i32, _i32, _p, _i64, ctypes.c_int, _p, _i32] + [_p] * 9 + [_sz, _p]
    L.gmi_moe_route_bwd.restype = ctypes.c_int
    L.gmi_moe_route_bwd.argtypes = [_i32, _i32, _i32, _p, _i64, ctypes.c_int, _p, _i32] + [_p] * 7 + [_i64, _p]
    L.gmi_group_rows_workspace_bytes.restype = _sz
    L.gmi_group_rows_workspace_bytes.argtypes = [_i32] * 2
    L.gmi_group_rows.restype = ctypes.c_int
    L.gmi_group_rows.argtypes = [_i32, _i32] + [_p] * 5 + [_sz, _p]
    L.gmi_moe_permute.restype = ctypes.c_int
    L.gmi_moe_permute.argtypes = [_i32, _i32, _i32, ctypes.c_int, _p, _i64, _p, _i64, _p, _i32, _p, _i64, _p, _i64, _p]
    L.gmi_moe_unpermute.restype = ctypes.c_int
    L.gmi_moe_unpermute.argtypes = [_i32, _i32, _i32, ctypes.c_int, _p, _i64, _i32, _p, _p, _p, _i64, _p, _i64, _p]
    L.gmi_moe_unpermute_bwd.restype = ctypes.c_int
    L.gmi_moe_unpermute_bwd.argtypes = [_i32, _i32, _i32, ctypes.c_int, _p, _i64, _p, _p, _p, _i64, _i32, _p, _i64, _p,
                                        _i64, _p, _i64, _p, _p]
    L.gmi_swiglu_quant.restype = ctypes.c_int
    L.gmi_swiglu_quant.argtypes = [_i32, _i32, ctypes.c_int, _p, _i64, _p, _p, _i64, _p, _i64, _p, _i64, _p]
    L.gmi_swiglu_bwd.restype = ctypes.c_int
    L.gmi_swiglu_bwd.argtypes = [_i32, _i32, ctypes.c_int, _p, _i64, _p, _i64, _p, _p, _i64, _p, _i64, _p, _i64, _p]
    L.gmi_gemm_lora_workspace_bytes.restype = _sz
    L.gmi_gemm_lora_workspace_bytes.argtypes = [_i32] * 4
    L.gmi_gemm_lora.restype = ctypes.c_int
    L.gmi_gemm_lora.argtypes = [_i32] * 5 + [ctypes.c_int, _p, _i64, _p, _i64, _i64, _p, _i64, _i64, _p, _p, _p, _p,
                                             _i64, _p, _i64, _p, _sz, _p]
    _lib = L
    return L


def _check(status: int) -> None:
    if status != GMI_OK:
        raise GmiError(status, lib().gmi_last_error().decode())


def _stream(stream) -> int:
    if stream is None:  # torch.cuda.current_stream().cuda_stream without the Stream object (2.8 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_on(stream, device: int) -> int:
    """The stream of a call whose tensors are on `device`: a kernel is launched on the current device."""
    current = torch._C._cuda_getDevice()
    if device != current:
        raise ValueError(f"the tensors are on device {device}, the current one is {current}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(current)
    at = getattr(stream, "device_index", None)
    if at is not None and at != device:
        raise ValueError(f"the tensors are on device {device}, the stream on {at}")
    return _stream(stream)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _ld(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit stride along its rows")
    return t.stride(0)


# ---------------------------------------------------------------- grouped
def time_next_gemm(start, stop) -> None:
    """Let the next GEMM kernel launched on this thread (grouped, grouped-offsets or pointer-array call) record
    `start` and `stop` around itself, so start.elapsed_time(stop) is that kernel's execution time.  Both are
    torch.cuda.Event(enable_timing=True) objects that have been recorded once (torch creates the HIP event on
    its first record); None, None cancels a pending request."""
    if start is None and stop is None:
        _check(lib().gmi_time_next_gemm(None, None))
        return
    _check(lib().gmi_time_next_gemm(start.cuda_event, stop.cuda_event))


def workspace_bytes(count: int) -> int:
    return lib().gmi_workspace_bytes(count)


def make_problems(As, Bs, Cs, Ds) -> "ctypes.Array":
    """gmi_problem array from lists of tensors: A [M][K], B [N][K] (column-major
    B, i.e. row n of the tensor is column n), C / D [M][N] (C may be None)."""
    arr = (Problem * len(As))()
    for i, (a, b, c, d) in enumerate(zip(As, Bs, Cs, Ds)):
        M, N = d.shape
        K = a.shape[1]
        arr[i] = Problem(M, N, K, _ld(a), _ld(b), _ld(c) if c is not None else 0, _ld(d),
                         _ptr(a), _ptr(b), _ptr(c), _ptr(d))
    return arr


def gemm_grouped(As, Bs, Cs, Ds, alpha=1.0, beta=0.0, workspace=None, stream=None):
    """D_g = alpha A_g B_g + beta C_g for every g, in one launch.  The element type is that of A
    (float8_e4m3fn A and B give bfloat16 C and D)."""
    dt = _DT[As[0].dtype]
    probs = make_problems(As, Bs, Cs if Cs is not None else [None] * len(As), Ds)
    need = workspace_bytes(len(As))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=Ds[0].device)
    _check(lib().gmi_gemm_grouped(probs, len(As), dt, alpha, beta, workspace.data_ptr(), workspace.numel(),
                                  _stream(stream)))
    return Ds


def gemm_grouped_raw(problems, count, dtype, alpha, beta, workspace, stream=None):
    """Call with a prepared gmi_problem array (no per-call marshalling)."""
    _check(lib().gmi_gemm_grouped(problems, count, dtype, alpha, beta, workspace.data_ptr(), workspace.numel(),
                                  _stream(stream)))


def _offsets_args(offsets, A, B, D):
    if B.dim() != 3 or B.stride(2) != 1 or B.stride(1) < B.shape[2]:
        raise ValueError("B must be [groups][N][K] with unit stride along K")
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int32 vector")
    count = B.shape[0]
    if offsets.numel() != count + 1:
        raise ValueError(f"offsets has {offsets.numel()} entries, {count + 1} expected")
    rows, N = D.shape
    K = A.shape[1]
    if A.shape[0] != rows or B.shape[1] != N or B.shape[2] != K:
        raise ValueError("A [rows][K], B [groups][N][K] and D [rows][N] disagree")
    return count, rows, N, K


def gemm_grouped_offsets(offsets: torch.Tensor, A: torch.Tensor, B: torch.Tensor, D: torch.Tensor,
                         C: torch.Tensor | None = None, alpha=1.0, beta=0.0, workspace=None, stream=None):
    """Grouped GEMM with device-held group sizes: group g owns rows offsets[g] .. offsets[g+1] of A [rows][K]
    and D [rows][N] (and C) and multiplies them by B[g] (B is [groups][N][K], each B[g] column-major K x N).
    `offsets` is a device int32 tensor of groups + 1 entries; nothing is read back to the host."""
    count, rows, N, K = _offsets_args(offsets, A, B, D)
    if workspace is None:
        workspace = torch.empty(workspace_bytes(count), dtype=torch.uint8, device=D.device)
    _check(lib().gmi_gemm_grouped_offsets(count, offsets.data_ptr(), rows, N, K, A.data_ptr(), _ld(A),
                                          B.data_ptr(), B.stride(1), B.stride(0), _ptr(C),
                                          _ld(C) if C is not None else 0, D.data_ptr(), _ld(D), _DT[A.dtype],
                                          alpha, beta, workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return D


def gemm_grouped_offsets_noalloc(offsets: torch.Tensor, A: torch.Tensor, B: torch.Tensor, D: torch.Tensor,
                                 C: torch.Tensor | None = None, alpha=1.0, beta=0.0, stream=None):
    """gemm_grouped_offsets without a workspace: the library keeps the group table in its own static device
    array (at most 1024 groups); calls that overlap on one device race on that array."""
    count, rows, N, K = _offsets_args(offsets, A, B, D)
    _check(lib().gmi_gemm_grouped_offsets_noalloc(count, offsets.data_ptr(), rows, N, K, A.data_ptr(), _ld(A),
                                                  B.data_ptr(), B.stride(1), B.stride(0), _ptr(C),
                                                  _ld(C) if C is not None else 0, D.data_ptr(), _ld(D), _DT[A.dtype],
                                                  alpha, beta, _stream(stream)))
    return D


# ---------------------------------------------------------------- ptr-array
def pointer_array(tensors, device) -> torch.Tensor:
    """Device array (int64) of the tensors' device addresses."""
    return torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64, device=device)


def gemm_ptr_array(L, M, N, K, A_ptrs, lda, B_ptrs, ldb, C_ptrs, ldc, D_ptrs, ldd, dtype, alpha=1.0, beta=0.0,
                   stream=None):
    """Pointer-array GEMM; *_ptrs are device int64 tensors of L addresses."""
    _check(lib().gmi_gemm_ptr_array(L, M, N, K, _ptr(A_ptrs), lda, _ptr(B_ptrs), ldb, _ptr(C_ptrs), ldc,
                                    _ptr(D_ptrs), ldd, _DT[dtype] if dtype in _DT else dtype, alpha, beta,
                                    _stream(stream)))


# ---------------------------------------------------------------- W4A16
def prepack_w4(w_u4: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Prepack a uint4 weight stored [N][K/2] (uint8) into the kernels' order."""
    if out is None:
        out = torch.empty(lib().gmi_prepack_w4_bytes(N, K), dtype=torch.uint8, device=w_u4.device)
    _check(lib().gmi_prepack_w4(w_u4.data_ptr(), N, K, out.data_ptr(), _stream(stream)))
    return out


def w4a16_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib().gmi_w4a16_workspace_bytes(M, N, K)


def gemm_w4a16(X: torch.Tensor, w_prepacked: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
               group_size: int, N: int, Y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Y = X W^T with X fp16 [M][K], scales fp16 [K/g][N], zeros uint8 [K/g][N/2].  `workspace` (a device
    byte tensor of at least w4a16_workspace_bytes(M, N, K)) enables the split-K path; pass an empty tensor
    (numel 0) to run unsplit.  With None, one is allocated for this call."""
    M, K = X.shape
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float16, device=X.device)
    if workspace is None:
        need = w4a16_workspace_bytes(M, N, K)
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    _check(lib().gmi_gemm_w4a16(M, N, K, X.data_ptr(), _ld(X), w_prepacked.data_ptr(), scales.data_ptr(),
                                zeros.data_ptr(), group_size, Y.data_ptr(), _ld(Y),
                                workspace.data_ptr() if workspace.numel() else None, workspace.numel(),
                                _stream(stream)))
    return Y


W4_TYPES = {"uint4": 0, "int4": 1}


def gemm_mixed(X: torch.Tensor, w_prepacked: torch.Tensor, scales: torch.Tensor | None, zeros: torch.Tensor | None,
               group_size: int, N: int, w_type: str = "uint4", Y: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X W^T in any conversion mode: scales None is the direct conversion, zeros None the conversion
    without zero point.  X, scales and Y share one type (float16 or bfloat16); `w_type` is "uint4" or
    "int4" (zero points, if any, have the same type).  Workspace as for gemm_w4a16."""
    M, K = X.shape
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    if workspace is None:
        workspace = torch.empty(w4a16_workspace_bytes(M, N, K), dtype=torch.uint8, device=X.device)
    _check(lib().gmi_gemm_mixed(M, N, K, _DT[X.dtype], X.data_ptr(), _ld(X), w_prepacked.data_ptr(),
                                W4_TYPES[w_type], _ptr(scales), _ptr(zeros), group_size, Y.data_ptr(), _ld(Y),
                                workspace.data_ptr() if workspace.numel() else None, workspace.numel(),
                                _stream(stream)))
    return Y


def gemm_mixed_grouped(offsets: torch.Tensor, X: torch.Tensor, w_prepacked: torch.Tensor,
                       scales: torch.Tensor | None, zeros: torch.Tensor | None, group_size: int, N: int,
                       w_type: str = "uint4", Y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Per-group Y_g = X_g W_g^T (mixture of experts): rows offsets[g] .. offsets[g+1] of X [rows][K] and Y
    [rows][N]; w_prepacked [groups][N*K/2] (each row a gmi_prepack_w4 output), scales [groups][K/g][N] or
    None, zeros [groups][K/g][N/2] or None.  `offsets` is a device int32 tensor of groups + 1 entries."""
    rows, K = X.shape
    count = w_prepacked.shape[0]
    if offsets.dtype != torch.int32 or offsets.numel() != count + 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int32 vector of groups + 1 entries")
    if Y is None:
        Y = torch.empty((rows, N), dtype=X.dtype, device=X.device)
    _check(lib().gmi_gemm_mixed_grouped(count, offsets.data_ptr(), rows, N, K, _DT[X.dtype], X.data_ptr(), _ld(X),
                                        w_prepacked.data_ptr(), w_prepacked.stride(0), W4_TYPES[w_type],
                                        _ptr(scales), scales.stride(0) if scales is not None else 0, _ptr(zeros),
                                        zeros.stride(0) if zeros is not None else 0, group_size, Y.data_ptr(),
                                        _ld(Y), _stream(stream)))
    return Y


# ---------------------------------------------------------------- conv
def conv_out_size(H, R, pad, stride, dil):
    return (H + 2 * pad - dil * (R - 1) - 1) // stride + 1


ACTIVATIONS = {None: 0, "none": 0, "relu": 1}


def conv2d_fprop(x: torch.Tensor, w: torch.Tensor, pad=(0, 0), stride=(1, 1), dil=(1, 1), c_in=None, alpha=1.0,
                 beta=0.0, y: torch.Tensor | None = None, stream=None, bias: torch.Tensor | None = None,
                 act: str | None = None) -> torch.Tensor:
    """Implicit-GEMM cross-correlation: x NHWC, w KRSC -> y NPQK.  With `bias` (K elements of x's type) or
    `act` ("relu"), the fused entry point adds the bias per output channel and applies the activation before
    the output is rounded."""
    N, H, W, C = x.shape
    K, R, S, _ = w.shape
    if y is None:
        P = conv_out_size(H, R, pad[0], stride[0], dil[0])
        Q = conv_out_size(W, S, pad[1], stride[1], dil[1])
        y = torch.empty((N, max(P, 0), max(Q, 0), K), dtype=x.dtype, device=x.device)
    if bias is None and act in (None, "none"):
        _check(lib().gmi_conv2d_fprop_implicit(N, H, W, C, K, R, S, pad[0], pad[1], stride[0], stride[1], dil[0],
                                               dil[1], x.data_ptr(), w.data_ptr(), _ptr(c_in), y.data_ptr(),
                                               _DT[x.dtype], alpha, beta, _stream(stream)))
    else:
        if bias is not None and (bias.numel() != K or bias.dtype != x.dtype):
            raise ValueError("bias must hold K elements of the activation's type")
        _check(lib().gmi_conv2d_fprop_implicit_fused(N, H, W, C, K, R, S, pad[0], pad[1], stride[0], stride[1],
                                                     dil[0], dil[1], x.data_ptr(), w.data_ptr(), _ptr(c_in),
                                                     _ptr(bias), y.data_ptr(), _DT[x.dtype], alpha, beta,
                                                     ACTIVATIONS[act], _stream(stream)))
    return y


def conv2d_dgrad(dy: torch.Tensor, w: torch.Tensor, H: int, W: int, pad=(0, 0), dil=(1, 1), c_in=None, alpha=1.0,
                 beta=0.0, dx: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stride=(1, 1),
                 stream=None) -> torch.Tensor:
    """Data gradient of conv2d_fprop: dy NPQK, w KRSC, the forward input's H, W -> dx NHWC (strides 1 .. 8 in
    each dimension)."""
    N, P, Q, K = dy.shape
    K2, R, S, C = w.shape
    if K2 != K:
        raise ValueError("dy and w disagree on K")
    if dx is None:
        dx = torch.empty((N, H, W, C), dtype=dy.dtype, device=dy.device)
    if workspace is None:
        workspace = torch.empty(lib().gmi_conv2d_dgrad_workspace_bytes(C, K, R, S), dtype=torch.uint8,
                                device=dy.device)
    _check(lib().gmi_conv2d_dgrad_implicit(N, H, W, C, K, R, S, pad[0], pad[1], stride[0], stride[1], dil[0], dil[1],
                                           dy.data_ptr(), w.data_ptr(), _ptr(c_in), dx.data_ptr(), _DT[dy.dtype],
                                           alpha, beta, workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return dx


def conv2d_wgrad_workspace_bytes(x_shape, dy_shape, R, S, pad=(0, 0), stride=(1, 1), dil=(1, 1), groups=1) -> int:
    N, H, W, C = x_shape
    K = dy_shape[3]
    return lib().gmi_conv2d_wgrad_workspace_bytes(N, H, W, C, K, R, S, pad[0], pad[1], stride[0], stride[1], dil[0],
                                                  dil[1], groups)


def conv2d_wgrad(x: torch.Tensor, dy: torch.Tensor, R: int, S: int, pad=(0, 0), stride=(1, 1), dil=(1, 1),
                 c_in=None, alpha=1.0, beta=0.0, dw: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, groups: int = 1, stream=None) -> torch.Tensor:
    """Filter gradient of conv2d_fprop: x NHWC, dy NPQK, the filter size R, S -> dw K x R x S x C/groups."""
    N, H, W, C = x.shape
    K = dy.shape[3]
    if dw is None:
        dw = torch.empty((K, R, S, C // groups), dtype=x.dtype, device=x.device)
    if workspace is None:
        workspace = torch.empty(conv2d_wgrad_workspace_bytes(x.shape, dy.shape, R, S, pad, stride, dil, groups),
                                dtype=torch.uint8, device=x.device)
    _check(lib().gmi_conv2d_wgrad_implicit(N, H, W, C, K, R, S, pad[0], pad[1], stride[0], stride[1], dil[0], dil[1],
                                           groups, x.data_ptr(), dy.data_ptr(), _ptr(c_in), dw.data_ptr(),
                                           _DT[x.dtype],
                                           alpha, beta, workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return dw


# ---------------------------------------------------------------- block-scaled fp8 mixture-of-experts layer
BLOCK = 128  # columns (and weight rows) per scale


def _scale_blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _new(shape, dtype, device, stream, returned=True) -> torch.Tensor:
    """A tensor this call makes, from the memory of the stream that the call runs on: memory let go on another stream
    may still be in use there.  A tensor that is returned is used and let go by the caller's current stream as well,
    so the allocator hears of that one too."""
    if stream is None or _stream(stream) == _stream(None):
        return torch.empty(shape, dtype=dtype, device=device)
    s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(s):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream())
    return t


_native = None


def _bound():
    """The native marshalling of the calls below, bound to the loaded libgmi.so.  It checks types, shapes, strides and
    devices (ValueError) and returns the library's status."""
    global _native
    if _native is None:
        L = lib()
        try:
            from . import _calls as native
        except ImportError as e:
            raise RuntimeError("the module _calls is not built; run __graft_entry__.build() or "
                               "python -m grouped_mixed_input_amd.build") from e
        native.bind(*(ctypes.cast(f, _p).value for f in (
            L.gmi_rmsnorm_quant, L.gmi_rmsnorm_bwd, L.gmi_gemm_f8_block, L.gmi_gemm_f8_block_grouped, L.gmi_moe_route,
            L.gmi_moe_route_bwd)), _stream)
        native.bind_rows(*(ctypes.cast(f, _p).value for f in (
            L.gmi_group_rows, L.gmi_moe_permute, L.gmi_moe_unpermute, L.gmi_moe_unpermute_bwd, L.gmi_swiglu_quant,
            L.gmi_swiglu_bwd, L.gmi_gemm_lora)), _stream_on)
        _native = native
    return _native


def _scratch(need: int, device, stream):
    """A workspace made for one call (None without need); the memory is reused in stream order."""
    return _new((need,), torch.uint8, device, stream, returned=False) if need else None


def rmsnorm_quant(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                  h: torch.Tensor | None = None, y: torch.Tensor | None = None, q: torch.Tensor | None = None,
                  scales: torch.Tensor | None = None, quantize: bool = True, stream=None):
    """h = x + residual; v = weight * h / sqrt(mean(h^2) + eps); q = e4m3(v / s) with one fp32 scale s per row and
    128 columns.  x [rows][K] float16 or bfloat16.  `h` (the sum, in x's type; may be x or residual) and `y` (v in
    x's type) are written where given.  Returns (q, scales), float8_e4m3fn [rows][K] and float32
    [rows][ceil(K / 128)]; with quantize=False only `y` (made if not given) is written and returned."""
    if quantize:
        if q is None:
            q = _new(x.shape, torch.float8_e4m3fn, x.device, stream)
        if scales is None:
            scales = _new((x.shape[0], _scale_blocks(x.shape[1])), torch.float32, x.device, stream)
    elif q is not None or scales is not None:
        raise ValueError("q and scales are written with quantize=True only")
    elif y is None:
        y = _new(x.shape, x.dtype, x.device, stream)
    _check(_bound().rmsnorm_quant(x, weight, residual, eps, h, y, q, scales, stream))
    return (q, scales) if quantize else y


def rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, dres: torch.Tensor | None = None,
                eps: float = 1e-6, dh: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None, weight_grad: bool = True):
    """Gradients of rmsnorm_quant's norm: `dy` is that of v, `h` the sum the forward wrote, `dres` the gradient that
    reaches h past the norm.  Returns (dh, dweight): dh in h's type (the gradient of x and of residual), dweight
    float32 [K].  With weight_grad=False (a frozen norm) dweight is None: one launch, and no workspace."""
    if dh is None:
        dh = _new(h.shape, h.dtype, h.device, stream)
    if weight_grad:
        if dweight is None:
            dweight = _new((h.shape[1],), torch.float32, h.device, stream)
        if workspace is None:
            workspace = _scratch(lib().gmi_rmsnorm_bwd_workspace_bytes(*h.shape), h.device, stream)
    elif dweight is not None:
        raise ValueError("dweight is written with weight_grad=True only")
    _check(_bound().rmsnorm_bwd(dy, h, weight, dres, eps, dh, dweight, workspace, stream))
    return dh, dweight


def _f8_out(rows: int, N: int, device, stream) -> torch.Tensor:
    return _new((rows, (N + 7) // 8 * 8), torch.bfloat16, device, stream)[:, :N]


def gemm_f8_block(X: torch.Tensor, x_scales: torch.Tensor, W: torch.Tensor, w_scales: torch.Tensor,
                  Y: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X W^T over block-scaled fp8: X float8_e4m3fn [M][K] with x_scales float32 [M][ceil(K / 128)], W
    float8_e4m3fn [N][K] with w_scales float32 [ceil(N / 128)][ceil(K / 128)]; Y bfloat16 [M][N].  `workspace` as
    for gemm_w4a16 (an empty tensor runs unsplit)."""
    if Y is None:
        Y = _f8_out(X.shape[0], W.shape[0], X.device, stream)
    if workspace is None:
        need = lib().gmi_gemm_f8_block_workspace_bytes(X.shape[0], W.shape[0], X.shape[1])
        workspace = _scratch(need, X.device, stream)
    _check(_bound().gemm_f8_block(X, x_scales, W, w_scales, Y, workspace, stream))
    return Y


def gemm_f8_block_grouped(offsets: torch.Tensor, X: torch.Tensor, x_scales: torch.Tensor, W: torch.Tensor,
                          w_scales: torch.Tensor, Y: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gemm_f8_block per group: rows offsets[g] .. offsets[g + 1] of X and Y belong to group g with weight W[g] (W
    [groups][N][K]) and scales w_scales[g].  `offsets` is a device int32 tensor of groups + 1 entries, as moe_route
    writes it; rows outside every group are not written."""
    if W.dim() != 3:
        raise ValueError("W must be [groups][N][K]")
    if Y is None:
        Y = _f8_out(X.shape[0], W.shape[1], X.device, stream)
    if W.shape[0] == 0:
        return Y
    if workspace is None:
        workspace = _scratch(lib().gmi_gemm_f8_block_grouped_workspace_bytes(W.shape[0]), X.device, stream)
    _check(_bound().gemm_f8_block_grouped(offsets, X, x_scales, W, w_scales, Y, workspace, stream))
    return Y


class Routing(NamedTuple):
    """What moe_route writes, int32 unless said otherwise: the experts of each token and their float32 weights
    [tokens][k], rows per expert, the row offsets [experts + 1] of the grouped calls, the row of each slot
    [tokens][k], the slot of each row [tokens * k], the balance loss (float32 [1]) and the live tokens [1]."""
    indices: torch.Tensor
    weights: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    slot_row: torch.Tensor
    row_slot: torch.Tensor
    loss: torch.Tensor
    live: torch.Tensor


def moe_route(logits: torch.Tensor, k: int, mask: torch.Tensor | None = None, renormalize: bool = True,
              out: Routing | None = None, workspace: torch.Tensor | None = None, stream=None) -> Routing:
    """Top-k routing of logits [tokens][experts] with the balance loss; see Routing.  `mask` (bool or uint8
    [tokens]) leaves tokens out: their slots hold expert -1.  `out` receives the results where given."""
    if out is None:
        (T, E), dev, i32, f32 = logits.shape, logits.device, torch.int32, torch.float32
        out = Routing(_new((T, k), i32, dev, stream), _new((T, k), f32, dev, stream), _new((E,), i32, dev, stream),
                      _new((E + 1,), i32, dev, stream), _new((T, k), i32, dev, stream), _new((T * k,), i32, dev, stream),
                      _new((1,), f32, dev, stream), _new((1,), i32, dev, stream))
    if workspace is None:
        workspace = _scratch(lib().gmi_moe_route_workspace_bytes(*logits.shape), logits.device, stream)
    _check(_bound().moe_route(logits, k, mask, renormalize, *out, workspace, stream))
    return out


def moe_route_bwd(logits: torch.Tensor, indices: torch.Tensor, weights: torch.Tensor, offsets: torch.Tensor,
                  live: torch.Tensor, dweights: torch.Tensor, dloss: torch.Tensor, mask: torch.Tensor | None = None,
                  renormalize: bool = True, dlogits: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of moe_route's logits from `dweights` [tokens][k] (float32) and `dloss` (float32 [1], on the
    device), with what the forward call wrote; mask and renormalize as given to it."""
    if dlogits is None:
        dlogits = _new(logits.shape, logits.dtype, logits.device, stream)
    _check(_bound().moe_route_bwd(logits, indices, weights, offsets, live, dweights, dloss, mask, renormalize, dlogits,
                                  stream))
    return dlogits


# ---------------------------------------------------------------- rows between the experts' products
class Grouping(NamedTuple):
    """What group_rows writes, int32: the row offsets [groups + 1], the rows by group [n] (those of no group last) and
    each row's place among them, in the shape of the index (-1 for rows of no group)."""
    offsets: torch.Tensor
    order: torch.Tensor
    place: torch.Tensor


def group_rows(index: torch.Tensor, groups: int, out: Grouping | None = None, workspace: torch.Tensor | None = None,
               stream=None) -> Grouping:
    """Rows ordered by the number that each carries: `index` int32, of any shape, its rows counted in memory order; see
    Grouping.  With the experts of a router's slots [tokens][k] as index, offsets, order and place serve as moe_route's
    offsets, row_slot and slot_row; with the adapters of a batch's rows, order is that of gemm_lora.  A row whose
    number lies outside [0, groups) belongs to no group."""
    if out is None:
        n, dev, i32 = index.numel(), index.device, torch.int32
        out = Grouping(_new((groups + 1,), i32, dev, stream), _new((n,), i32, dev, stream),
                       _new(index.shape, i32, dev, stream))
    if workspace is None:
        workspace = _scratch(lib().gmi_group_rows_workspace_bytes(index.numel(), groups), index.device, stream)
    _check(_bound().group_rows(index, groups, *out, workspace, stream))
    return out


def moe_permute(x: torch.Tensor, slot_row: torch.Tensor, scales: torch.Tensor | None = None,
                out: torch.Tensor | None = None, out_scales: torch.Tensor | None = None, stream=None):
    """Each token's row copied to the rows of its slots: out[slot_row[t, i]] = x[t].  x [tokens][K] float16, bfloat16 or
    float8_e4m3fn, the last with its `scales` float32 [tokens][ceil(K / 128)] where given; slot_row int32 [tokens][k]
    as moe_route writes it.  Returns out [tokens * k][K] (or as given), with scales (out, out_scales).  Rows that no
    slot has are not written.  The gradient is moe_unpermute without weights."""
    rows = slot_row.numel() if out is None else out.shape[0]
    if out is None:
        out = _new((rows, x.shape[1]), x.dtype, x.device, stream)
    if scales is not None and out_scales is None:
        out_scales = _new((rows, scales.shape[1]), torch.float32, x.device, stream)
    _check(_bound().moe_permute(x, slot_row, scales, out, out_scales, stream))
    return out if scales is None else (out, out_scales)


def moe_unpermute(rows: torch.Tensor, slot_row: torch.Tensor, weights: torch.Tensor | None = None,
                  add: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = add[t] + sum_i weights[t, i] * rows[slot_row[t, i]], summed in float32 and rounded once: the experts'
    rows [n][K] (float16 or bfloat16) back to the tokens.  `weights` float32 [tokens][k] (None: 1), `add` [tokens][K]
    in the rows' type (out may be add).  Slots without a row add nothing."""
    if out is None:
        out = _new((slot_row.shape[0], rows.shape[1]), rows.dtype, rows.device, stream)
    _check(_bound().moe_unpermute(rows, slot_row, weights, add, out, stream))
    return out


def moe_unpermute_bwd(dout: torch.Tensor, slot_row: torch.Tensor, weights: torch.Tensor | None = None,
                      rows: torch.Tensor | None = None, drows: torch.Tensor | None = None,
                      scales: torch.Tensor | None = None, dweights: torch.Tensor | None = None,
                      quantize: bool = False, stream=None, row_grad: bool = True):
    """Gradients of moe_unpermute: drows[slot_row[t, i]] = weights[t, i] * dout[t], in dout's type or with
    quantize=True as float8_e4m3fn with `scales` float32 [n][ceil(K / 128)], and dweights[t, i] = <dout[t],
    rows[slot_row[t, i]]> float32 where `rows` (what the forward call read) is given.  Returns (drows, dweights), or
    (drows, scales, dweights) with quantize; dweights is None without rows.  Rows that no slot has are not written.
    With row_grad=False (nothing behind the rows is trained) drows and scales are None."""
    if rows is None and (dweights is not None or not row_grad):
        raise ValueError("dweights needs the rows of the forward call")
    if not row_grad:
        if drows is not None or scales is not None or quantize:
            raise ValueError("drows and scales are written with row_grad=True only")
        if dweights is None:
            dweights = _new(slot_row.shape, torch.float32, dout.device, stream)
        _check(_bound().moe_unpermute_bwd(dout, slot_row, weights, rows, None, None, None, dweights, stream))
        return None, dweights
    if scales is not None and not quantize:
        raise ValueError("scales are written with quantize=True only")
    n = slot_row.numel() if rows is None else rows.shape[0]
    if drows is None:
        drows = _new((n, dout.shape[1]), torch.float8_e4m3fn if quantize else dout.dtype, dout.device, stream)
    if quantize and scales is None:
        scales = _new((drows.shape[0], _scale_blocks(dout.shape[1])), torch.float32, dout.device, stream)
    if rows is not None and dweights is None:
        dweights = _new(slot_row.shape, torch.float32, dout.device, stream)
    _check(_bound().moe_unpermute_bwd(dout, slot_row, weights, rows, None if quantize else drows,
                                      drows if quantize else None, scales, dweights, stream))
    return (drows, scales, dweights) if quantize else (drows, dweights)


def swiglu_quant(a: torch.Tensor, live: torch.Tensor | None = None, y: torch.Tensor | None = None,
                 q: torch.Tensor | None = None, scales: torch.Tensor | None = None, quantize: bool = True, stream=None):
    """v = silu(gate) * up of a [rows][2 N] (gate first; float16 or bfloat16) between an expert's two products: q =
    e4m3(v / s) with one float32 scale s per row and 128 columns; `y` (v in a's type) is written where given.  `live`
    (int32 [1] on the device: offsets[-1:] of the routing) leaves the rows from there on alone.  Returns (q, scales);
    with quantize=False only `y` (made if not given) is written and returned."""
    rows, N = a.shape[0], a.shape[1] // 2
    if quantize:
        if q is None:
            q = _new((rows, N), torch.float8_e4m3fn, a.device, stream)
        if scales is None:
            scales = _new((rows, _scale_blocks(N)), torch.float32, a.device, stream)
    elif q is not None or scales is not None:
        raise ValueError("q and scales are written with quantize=True only")
    elif y is None:
        y = _new((rows, N), a.dtype, a.device, stream)
    _check(_bound().swiglu_quant(a, live, y, q, scales, stream))
    return (q, scales) if quantize else y


def swiglu_bwd(dact: torch.Tensor, a: torch.Tensor, live: torch.Tensor | None = None, da: torch.Tensor | None = None,
               scales: torch.Tensor | None = None, quantize: bool = False, stream=None):
    """Gradient of swiglu_quant's v: da [rows][2 N], that of the gate first, from `dact` [rows][N] and the forward's
    `a`; in a's type (da may be a), or with quantize=True as float8_e4m3fn with `scales` float32
    [rows][ceil(2 N / 128)].  Returns da, or (da, scales)."""
    if scales is not None and not quantize:
        raise ValueError("scales are written with quantize=True only")
    if da is None:
        da = _new(a.shape, torch.float8_e4m3fn if quantize else a.dtype, a.device, stream)
    if quantize and scales is None:
        scales = _new((a.shape[0], _scale_blocks(a.shape[1])), torch.float32, a.device, stream)
    _check(_bound().swiglu_bwd(dact, a, live, None if quantize else da, da if quantize else None, scales, stream))
    return (da, scales) if quantize else da


# ---------------------------------------------------------------- adapters
def gemm_lora(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, index: torch.Tensor,
              scales: torch.Tensor | None = None, order: torch.Tensor | None = None, base: torch.Tensor | None = None,
              Y: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y[m] = base[m] + scales[a] * (X[m] A[a]^T) B[a]^T with a = index[m]: low-rank adapters of many requests beside one
    dense product, whose result is `base` (Y may be base; None: zeros).  X [M][K], A [adapters][rank][K], B
    [adapters][N][rank], base and Y [M][N] share one type, float16 or bfloat16; index int32 [M], -1 for rows without an
    adapter; scales float32 [adapters] (None: 1).  `order` (int32 [M], group_rows(index, adapters).order) brings rows
    of one adapter together, for speed: rows in any order give the same results.  `workspace`: a device byte tensor of
    lib().gmi_gemm_lora_workspace_bytes(M, N, K, rank) bytes; made for the call if not given."""
    if Y is None:
        Y = _new((X.shape[0], B.shape[1]), X.dtype, X.device, stream)
    if workspace is None:
        need = lib().gmi_gemm_lora_workspace_bytes(X.shape[0], B.shape[1], X.shape[1], A.shape[1])
        workspace = _scratch(need, X.device, stream)
    _check(_bound().gemm_lora(X, A, B, index, scales, order, base, Y, workspace, stream))
    return Y
