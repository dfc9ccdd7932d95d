"""W4A16 group-quantized linear layer for NVIDIA B200 (sm_100a).

A thin ctypes binding over ``libawq_b200.so`` (C ABI: ``include/awq.h``).
Every step of the computation runs in the library's CUDA kernels; this
module only checks tensors, allocates output buffers with PyTorch and passes
raw device pointers and the current CUDA stream. There is no CPU fallback:
importing the binding fails loudly if the shared library cannot be loaded.

Functions (same names as the C entry points):
  awq_packed_size, awq_workspace_bytes, awq_workspace_init, awq_pack,
  awq_dequant, awq_w4a16_gemv, awq_w4a16_gemm, awq_linear,
  awq_linear_gemv_limit, awq_linear_launches, awq_linear_path, awq_check_bounded_wait,
  awq_get_status, awq_status_string, awq_w4a16_gemv_no_alloc,
  awq_get_status_no_alloc, and the W4A8-FP8
  variant awq_fp8_row_exponents, awq_fp8_quantize_x, awq_dequant_fp8,
  awq_w4a8_gemm. Between the linear layers: awq_rmsnorm, awq_rmsnorm_fp8,
  awq_silu_mul, awq_silu_mul_fp8, and the 8-bit key/value cache
  awq_kv8_workspace_bytes, awq_kv8_append, awq_kv8_attention.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# AWQ_B200_DEBUG=1 loads the debug build (every guarded device access checks
# its index range and records AWQ_ERR_BOUNDS instead of faulting).
DEBUG = os.environ.get("AWQ_B200_DEBUG", "") == "1"
LIB_PATH = os.path.join(_PKG, "libawq_b200_debug.so" if DEBUG else "libawq_b200.so")

GROUP = 128
GEMV_MAX_M = 32

STATUS_NAMES = {
    0: "AWQ_OK", 1: "AWQ_ERR_INVALID_ARG", 2: "AWQ_ERR_SHAPE", 3: "AWQ_ERR_ALIGNMENT", 4: "AWQ_ERR_WORKSPACE",
    5: "AWQ_ERR_UNSUPPORTED", 6: "AWQ_ERR_CUDA", 7: "AWQ_ERR_TIMEOUT", 8: "AWQ_ERR_NONFINITE", 9: "AWQ_ERR_BOUNDS",
}
globals().update({name: code for code, name in STATUS_NAMES.items()})

# Every symbol include/awq.h declares.
EXPORTS = ("awq_packed_size", "awq_workspace_bytes", "awq_workspace_init", "awq_pack", "awq_dequant",
           "awq_w4a16_gemv", "awq_w4a16_gemm", "awq_linear", "awq_linear_gemv_limit", "awq_get_status",
           "awq_status_string", "awq_w4a16_gemv_no_alloc", "awq_get_status_no_alloc", "awq_linear_launches",
           "awq_linear_path",
           "awq_check_bounded_wait",
           "awq_fp8_row_exponents", "awq_fp8_quantize_x", "awq_dequant_fp8", "awq_w4a8_gemm",
           "awq_rmsnorm", "awq_rmsnorm_fp8", "awq_silu_mul", "awq_silu_mul_fp8",
           "awq_kv8_workspace_bytes", "awq_kv8_append", "awq_kv8_attention")


class AwqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {awq_status_string(status)}")


class _PackedSizes(ctypes.Structure):
    _fields_ = [("qweight_bytes", ctypes.c_size_t), ("scales_bytes", ctypes.c_size_t),
                ("zeros_bytes", ctypes.c_size_t)]


class _Kv8Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
                ("blocks", ctypes.c_int64), ("heads", ctypes.c_int32), ("block_tokens", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class _Kv8Batch(ctypes.Structure):
    _fields_ = [("starts", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("seqs", ctypes.c_int64), ("table_width", ctypes.c_int64)]


def _build_module():
    """build.py loaded by path (importing it must not load the library)."""
    import importlib.util
    spec = importlib.util.spec_from_file_location("_awq_b200_build", os.path.join(_PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _load() -> ctypes.CDLL:
    # (Re)compile in-tree with nvcc when the library is missing or older than
    # its sources; a failed build raises, there is no fallback.
    _build_module().build(debug=DEBUG)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, ci, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.awq_packed_size.argtypes = [i64, i64, ci, ctypes.POINTER(_PackedSizes)]
    lib.awq_workspace_bytes.argtypes = [i64, i64, i64, ci]
    lib.awq_workspace_bytes.restype = sz
    lib.awq_workspace_init.argtypes = [vp, sz, vp]
    lib.awq_pack.argtypes = [vp, i64, i64, ci, vp, vp, vp, vp, sz, vp]
    lib.awq_dequant.argtypes = [vp, vp, vp, i64, i64, ci, vp, vp]
    for f in ("awq_w4a16_gemv", "awq_w4a16_gemm", "awq_linear"):
        getattr(lib, f).argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp, sz, vp]
    lib.awq_w4a16_gemv_no_alloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp]
    lib.awq_get_status_no_alloc.argtypes = [vp]
    lib.awq_linear_gemv_limit.argtypes = []
    lib.awq_linear_launches.argtypes = [i64, i64, i64, ci]
    lib.awq_linear_path.argtypes = [i64, i64, i64, ci]
    lib.awq_check_bounded_wait.argtypes = [vp, sz, ctypes.c_uint32, vp]
    lib.awq_get_status.argtypes = [vp, vp]
    lib.awq_fp8_row_exponents.argtypes = [vp, i64, i64, ci, vp, vp]
    lib.awq_fp8_quantize_x.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.awq_dequant_fp8.argtypes = [vp, vp, vp, vp, i64, i64, ci, vp, vp]
    lib.awq_w4a8_gemm.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, vp, sz, vp]
    cf = ctypes.c_float
    lib.awq_rmsnorm.argtypes = [vp, vp, vp, cf, vp, vp, i64, i64, vp]
    lib.awq_rmsnorm_fp8.argtypes = [vp, vp, vp, cf, vp, vp, vp, i64, i64, vp]
    lib.awq_silu_mul.argtypes = [vp, vp, i64, i64, vp]
    lib.awq_silu_mul_fp8.argtypes = [vp, vp, vp, i64, i64, vp]
    pc, pb = ctypes.POINTER(_Kv8Cache), ctypes.POINTER(_Kv8Batch)
    lib.awq_kv8_workspace_bytes.argtypes = [i64, i64, ci, ci, ci]
    lib.awq_kv8_workspace_bytes.restype = sz
    lib.awq_kv8_append.argtypes = [vp, i64, vp, i64, pc, pb, vp, sz, vp]
    lib.awq_kv8_attention.argtypes = [vp, i64, ci, cf, pc, pb, vp, vp, sz, vp]
    lib.awq_status_string.argtypes = [ci]
    lib.awq_status_string.restype = ctypes.c_char_p
    for f in EXPORTS:
        if f not in ("awq_workspace_bytes", "awq_kv8_workspace_bytes", "awq_status_string"):
            getattr(lib, f).restype = ci
    return lib


lib = _load()


def awq_status_string(status: int) -> str:
    return lib.awq_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise AwqError(status, where)


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def awq_packed_size(K: int, N: int, group: int = GROUP) -> tuple[int, int, int]:
    out = _PackedSizes()
    _check(lib.awq_packed_size(K, N, group, ctypes.byref(out)), "awq_packed_size")
    return out.qweight_bytes, out.scales_bytes, out.zeros_bytes


def awq_workspace_bytes(M: int, K: int, N: int, group: int = GROUP) -> int:
    return int(lib.awq_workspace_bytes(M, K, N, group))


def awq_workspace_init(workspace: torch.Tensor):
    _check(lib.awq_workspace_init(_dev(workspace, torch.uint8, "workspace"), workspace.numel(),
                                  _stream(workspace)), "awq_workspace_init")


def new_workspace(M: int, K: int, N: int, device, group: int = GROUP) -> torch.Tensor:
    """Allocate (with torch) and zero a workspace large enough for (M, K, N)."""
    nbytes = awq_workspace_bytes(M, K, N, group)
    if nbytes == 0:
        raise AwqError(AWQ_ERR_SHAPE, "awq_workspace_bytes")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    awq_workspace_init(ws)
    return ws


def awq_pack(w: torch.Tensor, workspace: torch.Tensor, group: int = GROUP):
    """w fp16 [N][K] -> (qweight int32 [(N/16)*(K/128)][16][16] packed blocks in the order
    include/awq.h documents, scales fp16 [K/G][N], zeros uint8 [K/G][N/2])."""
    N, K = w.shape
    qweight = torch.empty(((N // 16) * (K // 128), 16, 16), dtype=torch.int32, device=w.device)
    scales = torch.empty((K // group, N), dtype=torch.float16, device=w.device)
    zeros = torch.empty((K // group, N // 2), dtype=torch.uint8, device=w.device)
    _check(lib.awq_pack(_dev(w, torch.float16, "w"), K, N, group, qweight.data_ptr(), scales.data_ptr(),
                        zeros.data_ptr(), _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(w)),
           "awq_pack")
    return qweight, scales, zeros


def awq_dequant(qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, K: int, N: int,
                group: int = GROUP) -> torch.Tensor:
    w = torch.empty((N, K), dtype=torch.float16, device=qweight.device)
    _check(lib.awq_dequant(_dev(qweight, torch.int32, "qweight"), _dev(scales, torch.float16, "scales"),
                           _dev(zeros, torch.uint8, "zeros"), K, N, group, w.data_ptr(), _stream(qweight)),
           "awq_dequant")
    return w


def _linear_call(fn, name, x, qweight, scales, zeros, N, workspace, group, y):
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    elif y.shape != (M, N):
        raise ValueError(f"y must be [{M}, {N}]")
    _check(fn(_dev(x, torch.float16, "x"), _dev(qweight, torch.int32, "qweight"),
              _dev(scales, torch.float16, "scales"), _dev(zeros, torch.uint8, "zeros"),
              _dev(y, torch.float16, "y"), M, K, N, group, _dev(workspace, torch.uint8, "workspace"),
              workspace.numel(), _stream(x)), name)
    return y


def awq_w4a16_gemv(x, qweight, scales, zeros, N, workspace, group: int = GROUP, y=None):
    """Decode GEMV (1 <= M <= 32): y fp16 [M][N] = x fp16 [M][K] . W^T."""
    return _linear_call(lib.awq_w4a16_gemv, "awq_w4a16_gemv", x, qweight, scales, zeros, N, workspace, group, y)


def awq_w4a16_gemm(x, qweight, scales, zeros, N, workspace, group: int = GROUP, y=None):
    """Prefill GEMM on tcgen05 tensor cores (any M)."""
    return _linear_call(lib.awq_w4a16_gemm, "awq_w4a16_gemm", x, qweight, scales, zeros, N, workspace, group, y)


def awq_linear(x, qweight, scales, zeros, N, workspace, group: int = GROUP, y=None):
    """The linear layer: the GEMV for M <= awq_linear_gemv_limit() (and up to
    M = 32 on layers with fewer 128-channel tiles than SMs), the GEMM otherwise."""
    return _linear_call(lib.awq_linear, "awq_linear", x, qweight, scales, zeros, N, workspace, group, y)


def awq_w4a16_gemv_no_alloc(x, qweight, scales, zeros, N, group: int = GROUP, y=None):
    """Decode GEMV for callers that cannot allocate device memory: no
    workspace argument; the library's own static scratch array is used (see
    include/awq.h). Here torch allocates y only when the caller passes none."""
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    _check(lib.awq_w4a16_gemv_no_alloc(_dev(x, torch.float16, "x"), _dev(qweight, torch.int32, "qweight"),
                                       _dev(scales, torch.float16, "scales"), _dev(zeros, torch.uint8, "zeros"),
                                       _dev(y, torch.float16, "y"), M, K, N, group, _stream(x)),
           "awq_w4a16_gemv_no_alloc")
    return y


def awq_get_status_no_alloc(device=None) -> int:
    """Synchronize the current stream; return (and clear) the status word of
    the no-alloc GEMV's scratch array on the current device."""
    return int(lib.awq_get_status_no_alloc(torch.cuda.current_stream(device).cuda_stream))


def awq_fp8_row_exponents(scales: torch.Tensor, K: int, N: int, group: int = GROUP) -> torch.Tensor:
    """int8 [N]: per output channel, the power of two that moves its weights into
    the E4M3 range (W4A8-FP8 variant; once per weight, like awq_pack)."""
    e = torch.empty(N, dtype=torch.int8, device=scales.device)
    _check(lib.awq_fp8_row_exponents(_dev(scales, torch.float16, "scales"), K, N, group, e.data_ptr(),
                                     _stream(scales)), "awq_fp8_row_exponents")
    return e


def awq_fp8_quantize_x(x: torch.Tensor):
    """x fp16 [M][K] -> (x8 uint8 E4M3 codes [M][K], sx float32 [M])."""
    M, K = x.shape
    x8 = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    sx = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib.awq_fp8_quantize_x(_dev(x, torch.float16, "x"), M, K, x8.data_ptr(), sx.data_ptr(), _stream(x)),
           "awq_fp8_quantize_x")
    return x8, sx


def awq_dequant_fp8(qweight, scales, zeros, row_exp, K: int, N: int, group: int = GROUP) -> torch.Tensor:
    """uint8 [N][K]: the E4M3 weight codes the W4A8 GEMM multiplies (test surface)."""
    w8 = torch.empty((N, K), dtype=torch.uint8, device=qweight.device)
    _check(lib.awq_dequant_fp8(_dev(qweight, torch.int32, "qweight"), _dev(scales, torch.float16, "scales"),
                               _dev(zeros, torch.uint8, "zeros"), _dev(row_exp, torch.int8, "row_exp"), K, N, group,
                               w8.data_ptr(), _stream(qweight)), "awq_dequant_fp8")
    return w8


def awq_w4a8_gemm(x8, sx, qweight, scales, zeros, row_exp, N, workspace, group: int = GROUP, y=None):
    """W4A8-FP8 prefill GEMM (tcgen05 kind::f8f6f4): y fp16 [M][N] from the
    outputs of awq_fp8_quantize_x and awq_fp8_row_exponents."""
    M, K = x8.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x8.device)
    elif y.shape != (M, N):
        raise ValueError(f"y must be [{M}, {N}]")
    _check(lib.awq_w4a8_gemm(_dev(x8, torch.uint8, "x8"), _dev(sx, torch.float32, "sx"),
                             _dev(qweight, torch.int32, "qweight"), _dev(scales, torch.float16, "scales"),
                             _dev(zeros, torch.uint8, "zeros"), _dev(row_exp, torch.int8, "row_exp"),
                             _dev(y, torch.float16, "y"), M, K, N, group, _dev(workspace, torch.uint8, "workspace"),
                             workspace.numel(), _stream(x8)), "awq_w4a8_gemm")
    return y


# The current device and the raw handle of its current stream, without the
# Python objects around them (2 us a call) where torch has the short way.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


@functools.cache
def _device_count() -> int:
    return torch.cuda.device_count()


def _call(fn, name: str, tensors, *args):
    """fn(*args, stream) on the device of the tensors (which must share one),
    on that device's current stream."""
    device = tensors[0].get_device()
    if _device_count() > 1:  # every tensor is known to be on a GPU
        for t in tensors:
            if t.get_device() != device:
                raise ValueError(f"{name}: tensors on {tensors[0].device} and {t.device}")
    if device == _current_device():
        status = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device))
    if status != 0:
        raise AwqError(status, name)


def _empty(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """torch.empty((rows, cols)) by its shortest way (1.4 us against 2.3)."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _given(t, shape, dtype, name: str) -> torch.Tensor:
    """The caller's output `t`, checked."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    _dev(t, dtype, name)
    return t


def _norm_inputs(x, weight, residual, h):
    M, K = x.shape
    tensors = [x, weight]
    px, pw = _dev(x, torch.float16, "x"), _dev(weight, torch.float16, "weight")
    if weight.shape != (K,):
        raise ValueError(f"weight must be [{K}]")
    if residual is None:
        if h is not None:
            raise ValueError("h needs a residual")
        return M, K, tensors, px, None, pw, None
    pr = _dev(residual, torch.float16, "residual")
    if residual.shape != (M, K):
        raise ValueError(f"residual must be [{M}, {K}]")
    h = torch.empty_like(x) if h is None else _given(h, (M, K), torch.float16, "h")
    return M, K, tensors + [residual, h], px, pr, pw, h


def awq_rmsnorm(x, weight, eps: float, residual=None, h=None, y=None):
    """y fp16 [M][K] = n * rsqrt(mean(n^2) + eps) * weight with n = x, or with a
    residual n = x + residual; then (y, h) is returned, h = n rounded to fp16
    (h may be x or residual itself: updated in place)."""
    M, K, tensors, px, pr, pw, h = _norm_inputs(x, weight, residual, h)
    y = torch.empty_like(x) if y is None else _given(y, (M, K), torch.float16, "y")
    _call(lib.awq_rmsnorm, "awq_rmsnorm", tensors + [y], px, pr, pw, eps, None if h is None else h.data_ptr(),
          y.data_ptr(), M, K)
    return y if h is None else (y, h)


def awq_rmsnorm_fp8(x, weight, eps: float, residual=None, h=None, x8=None, sx=None):
    """awq_rmsnorm with y as (x8 uint8 E4M3 codes [M][K], sx float32 [M]), the
    inputs of awq_w4a8_gemm; (x8, sx, h) with a residual."""
    M, K, tensors, px, pr, pw, h = _norm_inputs(x, weight, residual, h)
    x8 = torch.empty_like(x, dtype=torch.uint8) if x8 is None else _given(x8, (M, K), torch.uint8, "x8")
    sx = x.new_empty(M, dtype=torch.float32) if sx is None else _given(sx, (M,), torch.float32, "sx")
    _call(lib.awq_rmsnorm_fp8, "awq_rmsnorm_fp8", tensors + [x8, sx], px, pr, pw, eps,
          None if h is None else h.data_ptr(), x8.data_ptr(), sx.data_ptr(), M, K)
    return (x8, sx) if h is None else (x8, sx, h)


def _gate_up(gate_up):
    M, F2 = gate_up.shape
    if F2 % 2:
        raise ValueError("gate_up must be [M, 2F]")
    return M, F2 // 2, _dev(gate_up, torch.float16, "gate_up")


def awq_silu_mul(gate_up, y=None):
    """gate_up fp16 [M][2F] -> y fp16 [M][F] = silu(gate_up[:, :F]) * gate_up[:, F:]."""
    M, F, p = _gate_up(gate_up)
    y = _empty(M, F, torch.float16, gate_up.device) if y is None else _given(y, (M, F), torch.float16, "y")
    _call(lib.awq_silu_mul, "awq_silu_mul", (gate_up, y), p, y.data_ptr(), M, F)
    return y


def awq_silu_mul_fp8(gate_up, x8=None, sx=None):
    """awq_silu_mul with y as (x8 uint8 E4M3 codes [M][F], sx float32 [M]), the
    inputs of awq_w4a8_gemm."""
    M, F, p = _gate_up(gate_up)
    x8 = _empty(M, F, torch.uint8, gate_up.device) if x8 is None else _given(x8, (M, F), torch.uint8, "x8")
    sx = gate_up.new_empty(M, dtype=torch.float32) if sx is None else _given(sx, (M,), torch.float32, "sx")
    _call(lib.awq_silu_mul_fp8, "awq_silu_mul_fp8", (gate_up, x8, sx), p, x8.data_ptr(), sx.data_ptr(), M, F)
    return x8, sx


class Kv8Cache(NamedTuple):
    """An 8-bit key/value cache: E4M3 codes uint8 [blocks][heads][block_tokens]
    [head_dim] and their exponents int8 [blocks][heads]; value = code * 2^exp."""
    k: torch.Tensor
    v: torch.Tensor
    k_exp: torch.Tensor
    v_exp: torch.Tensor


def new_kv8_cache(blocks: int, heads: int, block_tokens: int, head_dim: int, device) -> Kv8Cache:
    """Allocate (with torch) an empty cache."""
    codes = (blocks, heads, block_tokens, head_dim)
    return Kv8Cache(torch.zeros(codes, dtype=torch.uint8, device=device),
                    torch.zeros(codes, dtype=torch.uint8, device=device),
                    torch.zeros(codes[:2], dtype=torch.int8, device=device),
                    torch.zeros(codes[:2], dtype=torch.int8, device=device))


def awq_kv8_workspace_bytes(rows: int, seqs: int, q_heads: int, heads: int, head_dim: int) -> int:
    return int(lib.awq_kv8_workspace_bytes(rows, seqs, q_heads, heads, head_dim))


def new_kv8_workspace(rows: int, seqs: int, q_heads: int, heads: int, head_dim: int, device) -> torch.Tensor:
    """Allocate (with torch) and zero a workspace for awq_kv8_append and awq_kv8_attention."""
    with torch.cuda.device(device):
        nbytes = awq_kv8_workspace_bytes(rows, seqs, q_heads, heads, head_dim)
        if nbytes == 0:
            raise AwqError(AWQ_ERR_SHAPE, "awq_kv8_workspace_bytes")
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        awq_workspace_init(ws)
    return ws


def _kv8_rows(t, rows, heads, head_dim, name):
    """Pointer and row stride of fp16 [rows][heads][head_dim] whose rows may lie
    apart (a column range of a wider matrix)."""
    if not t.is_cuda or t.dtype != torch.float16:
        raise ValueError(f"{name} must be a CUDA tensor of torch.float16")
    if t.shape != (rows, heads, head_dim):
        raise ValueError(f"{name} must be [{rows}, {heads}, {head_dim}]")
    stride, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != head_dim):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), (stride if rows > 1 else heads * head_dim)


def _kv8_call(fn, name, rows, cache, starts, lens, table, workspace, tensors, before, after):
    k, v, k_exp, v_exp = cache
    shape = k.shape
    blocks, heads, block_tokens, head_dim = shape
    if v.shape != shape or k_exp.shape != (blocks, heads) or v_exp.shape != (blocks, heads):
        raise ValueError("cache parts must be [blocks, heads, block_tokens, head_dim] and [blocks, heads]")
    c = _Kv8Cache(_dev(k, torch.uint8, "cache.k"), _dev(v, torch.uint8, "cache.v"),
                  _dev(k_exp, torch.int8, "cache.k_exp"), _dev(v_exp, torch.int8, "cache.v_exp"), blocks, heads,
                  block_tokens, head_dim)
    seqs, width = table.shape
    if starts.shape != (seqs + 1,) or lens.shape != (seqs,):
        raise ValueError(f"starts must be [{seqs + 1}] and lens [{seqs}]")
    b = _Kv8Batch(_dev(starts, torch.int32, "starts"), _dev(lens, torch.int32, "lens"),
                  _dev(table, torch.int32, "block_table"), rows, seqs, width)
    _call(fn, name, (k, v, k_exp, v_exp, starts, lens, table, workspace, *tensors), *before, c, b, *after,
          _dev(workspace, torch.uint8, "workspace"), workspace.numel())


def awq_kv8_append(k, v, cache: Kv8Cache, starts, lens, block_table, workspace):
    """Write the new tokens' k and v, fp16 [rows][heads][head_dim], into the
    cache: sequence b owns rows starts[b] .. starts[b+1]-1, has lens[b] tokens
    with them (the last ones), and its token j lies in block
    block_table[b][j // block_tokens] (int32 tensors; see include/awq.h)."""
    _, heads, _, head_dim = cache[0].shape
    rows = k.shape[0]
    pk, sk = _kv8_rows(k, rows, heads, head_dim, "k")
    pv, sv = _kv8_rows(v, rows, heads, head_dim, "v")
    _kv8_call(lib.awq_kv8_append, "awq_kv8_append", rows, cache, starts, lens, block_table, workspace, (k, v),
              (pk, sk, pv, sv), ())


def awq_kv8_attention(q, cache: Kv8Cache, starts, lens, block_table, workspace, scale: float | None = None, y=None):
    """Causal attention of the new rows q fp16 [rows][q_heads][head_dim] over the
    cache (after awq_kv8_append, same starts, lens and block_table): y fp16
    [rows][q_heads * head_dim]. scale: 1 / sqrt(head_dim) unless given. Rows
    of y that belong to no sequence are not written."""
    rows, q_heads, head_dim = q.shape
    if head_dim != cache[0].shape[3]:
        raise ValueError(f"q must be [rows, q_heads, {cache[0].shape[3]}]")
    pq, sq = _kv8_rows(q, rows, q_heads, head_dim, "q")
    width = q_heads * head_dim
    y = _empty(rows, width, torch.float16, q.device) if y is None else _given(y, (rows, width), torch.float16, "y")
    _kv8_call(lib.awq_kv8_attention, "awq_kv8_attention", rows, cache, starts, lens, block_table, workspace, (q, y),
              (pq, sq, q_heads, head_dim ** -0.5 if scale is None else scale), (y.data_ptr(),))
    return y


def awq_linear_gemv_limit() -> int:
    return int(lib.awq_linear_gemv_limit())


def awq_linear_launches(M: int, K: int, N: int, group: int = GROUP) -> int:
    """Kernels awq_linear launches for these sizes on the current device."""
    return int(lib.awq_linear_launches(M, K, N, group))


def awq_linear_path(M: int, K: int, N: int, group: int = GROUP) -> int:
    """Kernel awq_linear runs for these sizes: 1 = the GEMV, 2 = the GEMM, 3 = the
    GEMM on CTA pairs, 0 = none."""
    return int(lib.awq_linear_path(M, K, N, group))


def awq_check_bounded_wait(workspace: torch.Tensor, limit_us: int = 1000):
    """Run the kernels' bounded wait on a barrier nothing completes (self-test);
    afterwards awq_get_status(workspace) reports AWQ_ERR_TIMEOUT."""
    _check(lib.awq_check_bounded_wait(_dev(workspace, torch.uint8, "workspace"), workspace.numel(), limit_us,
                                      _stream(workspace)), "awq_check_bounded_wait")


def awq_get_status(workspace: torch.Tensor) -> int:
    """Synchronize the current stream; return (and clear) the device-side status word."""
    return int(lib.awq_get_status(_dev(workspace, torch.uint8, "workspace"), _stream(workspace)))
