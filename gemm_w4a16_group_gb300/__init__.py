"""GB300 (sm_103a) W4A16 group-quantized matmul: thin Python binding.

Every call marshals torch tensors into the C ABI of ``include/w4a16.h`` and
runs on the current CUDA stream; all arithmetic happens in the CUDA library
(``_build/libw4a16_gb300.so``, built in-tree by ``build.py``). There is no
CPU or PyTorch fallback: if the library cannot be loaded every call raises.

    packed = repack(qweight, scales, zeros, N, K, group, sym)     # once per weight
    y = gemm(x, packed, N, K, group, sym)                          # y = x . dequant(W)^T
    pg = repack_gateup(qg, sg, zg, qu, su, zu, N, K, group, sym)
    h = gateup_silu(x, pg, N, K, group, sym)                       # SiLU(x Wg^T) * (x Wu^T)

Affine form w = scale * q + bias (MLX affine 4-bit checkpoints):

    pa = repack_affine(qweight, scales, biases, N, K, group)
    xs = xsum(x, K, group)                 # group sums of x, shared by every weight on x
    y = gemm_affine(x, pa, N, K, group, xs)

The rest of a verify step of drafted token trees over a paged key/value cache
(k_cache, v_cache [pages, kv heads, page rows, dim], bf16 or float8_e4m3fn):

    kv_reserve(table, refs, rows, want, page_rows)                 # pages for the new tokens
    kv_append(k, v, k_cache, v_cache, table, lengths, starts)      # per layer
    o = tree_attention(q, k_cache, v_cache, table, lengths, starts, mask, max_tree)
    path, count, token = tree_accept(target, draft, mask, starts, max_tree)
    lengths = kv_compact(k_layers, v_layers, table, lengths, path, count)
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct as _struct
import threading as _threading

from . import build as _build

__all__ = [
    "EXPORTS", "W4A16Error", "lib", "library_path", "repacked_bytes", "gateup_repacked_bytes",
    "repack", "repack_gateup", "gemm", "gemm_argmax", "gateup_silu", "dequantize", "kernel_status",
    "set_kernel_override", "set_programmatic_overlap", "strerror", "KERNEL_AUTO", "KERNEL_GEMV", "KERNEL_SMALLM", "KERNEL_TC",
    "KERNEL_XSTAGED", "KERNEL_DECODE_TC",
    "AFFINE", "repack_affine", "repack_affine_gateup", "xsum_bytes", "xsum", "gemm_affine", "gateup_silu_affine",
    "gemm_affine_noalloc", "topk", "gemm_topk", "affine_bits_repacked_bytes", "repack_affine_bits",
    "affine_bits_scratch_bytes", "gemm_affine_bits", "dequantize_affine_bits",
    "MAX_TREE", "MAX_ROWS", "kv_append", "tree_attention_workspace_bytes", "tree_attention", "tree_accept", "kv_compact",
    "kv_free", "kv_fork", "kv_reserve",
]

# symbols declared in include/w4a16.h
EXPORTS = (
    "w4a16_repacked_bytes", "w4a16_repack", "w4a16_gateup_repacked_bytes", "w4a16_repack_gateup",
    "w4a16_gemm", "w4a16_gemm_argmax", "w4a16_gateup_silu", "w4a16_dequantize", "w4a16_kernel_status",
    "w4a16_strerror", "w4a16_last_cuda_error", "w4a16_set_kernel_override",
    "w4a16_set_programmatic_overlap", "w4a16_repack_affine", "w4a16_repack_affine_gateup", "w4a16_xsum_bytes",
    "w4a16_xsum", "w4a16_gemm_affine", "w4a16_gateup_silu_affine", "w4a16_gemm_affine_noalloc",
    "w4a16_topk", "w4a16_gemm_topk", "w4a16_affine_bits_repacked_bytes", "w4a16_repack_affine_bits",
    "w4a16_affine_bits_scratch_bytes", "w4a16_gemm_affine_bits", "w4a16_dequantize_affine_bits",
    "w4a16_kv_append", "w4a16_tree_attention_workspace_bytes", "w4a16_tree_attention", "w4a16_tree_accept",
    "w4a16_kv_compact", "w4a16_kv_free", "w4a16_kv_fork", "w4a16_kv_reserve",
)
KERNEL_AUTO, KERNEL_GEMV, KERNEL_SMALLM, KERNEL_TC, KERNEL_XSTAGED, KERNEL_DECODE_TC = 0, 1, 2, 3, 4, 5
# the `sym` argument: 0 zero points, 1 symmetric (z = 8), AFFINE scale * q + bias
AFFINE = 2


class W4A16Error(RuntimeError):
    pass


_lib = None


def library_path() -> str:
    return _build.LIB


def lib(auto_build: bool = True) -> ctypes.CDLL:
    """The loaded CUDA library (compiled first if missing or stale and nvcc is present)."""
    global _lib
    if _lib is not None:
        return _lib
    if auto_build and not _build.up_to_date():
        try:
            _build.build()
        except Exception as e:  # fall through to the load error below
            if not os.path.exists(_build.LIB):
                raise W4A16Error(f"CUDA library missing and build failed: {e}") from e
    if not os.path.exists(_build.LIB):
        raise W4A16Error(f"CUDA library not built: {_build.LIB}")
    L = ctypes.CDLL(_build.LIB)
    P, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.w4a16_repacked_bytes.argtypes = [i32, i32, i32, i32]
    L.w4a16_repacked_bytes.restype = sz
    L.w4a16_gateup_repacked_bytes.argtypes = [i32, i32, i32, i32]
    L.w4a16_gateup_repacked_bytes.restype = sz
    L.w4a16_repack.argtypes = [P, P, P, i32, i32, i32, i32, P, P]
    L.w4a16_repack.restype = i32
    L.w4a16_repack_gateup.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, P, P]
    L.w4a16_repack_gateup.restype = i32
    L.w4a16_gemm.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, P, P]
    L.w4a16_gemm.restype = i32
    L.w4a16_gemm_argmax.argtypes = [P, P, i32, i32, i32, i32, i32, P, P, P]
    L.w4a16_gemm_argmax.restype = i32
    L.w4a16_gateup_silu.argtypes = [P, P, i32, i32, i32, i32, i32, P, P]
    L.w4a16_gateup_silu.restype = i32
    L.w4a16_dequantize.argtypes = [P, i32, i32, i32, i32, P, P]
    L.w4a16_dequantize.restype = i32
    L.w4a16_kernel_status.argtypes = []
    L.w4a16_kernel_status.restype = i32
    L.w4a16_strerror.argtypes = [i32]
    L.w4a16_strerror.restype = ctypes.c_char_p
    L.w4a16_last_cuda_error.argtypes = []
    L.w4a16_last_cuda_error.restype = i32
    L.w4a16_set_kernel_override.argtypes = [i32]
    L.w4a16_set_kernel_override.restype = i32
    L.w4a16_set_programmatic_overlap.argtypes = [i32]
    L.w4a16_set_programmatic_overlap.restype = i32
    L.w4a16_repack_affine.argtypes = [P, P, P, i32, i32, i32, P, P]
    L.w4a16_repack_affine.restype = i32
    L.w4a16_repack_affine_gateup.argtypes = [P, P, P, P, P, P, i32, i32, i32, P, P]
    L.w4a16_repack_affine_gateup.restype = i32
    L.w4a16_xsum_bytes.argtypes = [i32, i32, i32]
    L.w4a16_xsum_bytes.restype = sz
    L.w4a16_xsum.argtypes = [P, i32, i32, i32, P, P]
    L.w4a16_xsum.restype = i32
    L.w4a16_gemm_affine.argtypes = [P, P, P, i32, i32, i32, i32, P, P]
    L.w4a16_gemm_affine.restype = i32
    L.w4a16_gateup_silu_affine.argtypes = [P, P, P, i32, i32, i32, i32, P, P]
    L.w4a16_gateup_silu_affine.restype = i32
    L.w4a16_gemm_affine_noalloc.argtypes = [P, P, i32, i32, i32, i32, P, P]
    L.w4a16_gemm_affine_noalloc.restype = i32
    L.w4a16_topk.argtypes = [P, i32, i32, i32, P, P, P]
    L.w4a16_topk.restype = i32
    L.w4a16_gemm_topk.argtypes = [P, P, i32, i32, i32, i32, i32, i32, P, P, P, P]
    L.w4a16_gemm_topk.restype = i32
    L.w4a16_affine_bits_repacked_bytes.argtypes = [i32, i32, i32, i32]
    L.w4a16_affine_bits_repacked_bytes.restype = ctypes.c_size_t
    L.w4a16_repack_affine_bits.argtypes = [P, P, P, i32, i32, i32, i32, P, P]
    L.w4a16_repack_affine_bits.restype = i32
    L.w4a16_affine_bits_scratch_bytes.argtypes = [i32, i32, i32, i32]
    L.w4a16_affine_bits_scratch_bytes.restype = ctypes.c_size_t
    L.w4a16_gemm_affine_bits.argtypes = [P, P, P, i32, i32, i32, i32, i32, P, P]
    L.w4a16_gemm_affine_bits.restype = i32
    L.w4a16_dequantize_affine_bits.argtypes = [P, i32, i32, i32, i32, P, P]
    L.w4a16_dequantize_affine_bits.restype = i32
    i64, f32 = ctypes.c_int64, ctypes.c_float
    L.w4a16_kv_append.argtypes = [P, P, i64, i64, i64, i64, P, P, i32, P, P, i32, i32, P]
    L.w4a16_kv_append.restype = i32
    L.w4a16_tree_attention_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.w4a16_tree_attention_workspace_bytes.restype = sz
    L.w4a16_tree_attention.argtypes = [P, i64, i64, P, P, i32, P, P, P, i32, i32, i32, i32, f32, P, P, P]
    L.w4a16_tree_attention.restype = i32
    L.w4a16_tree_accept.argtypes = [P, P, P, P, i32, i32, i32, P, P, P, P]
    L.w4a16_tree_accept.restype = i32
    L.w4a16_kv_compact.argtypes = [P, P, i32, P, P, P, i32, i32, P, P]
    L.w4a16_kv_compact.restype = i32
    L.w4a16_kv_free.argtypes = [P, i32, i32, P, P, i32, P, i32, P]
    L.w4a16_kv_free.restype = i32
    L.w4a16_kv_fork.argtypes = [P, P, i32, i32, P, P, P, P, i32, P, P]
    L.w4a16_kv_fork.restype = i32
    L.w4a16_kv_reserve.argtypes = [P, i32, i32, P, i32, i32, P, P, i32, P, P]
    L.w4a16_kv_reserve.restype = i32
    _lib = L
    return L


def strerror(rc: int) -> str:
    return lib().w4a16_strerror(rc).decode()


def _check(rc: int, what: str):
    if rc != 0:
        msg = f"{what}: {strerror(rc)} (status {rc}"
        if rc == -4:
            msg += f", cudaError {lib().w4a16_last_cuda_error()}"
        raise W4A16Error(msg + ")")


def _torch():
    import torch
    return torch


@functools.lru_cache(maxsize=1)
def _device_count() -> int:
    return _torch().cuda.device_count()


def _stream(stream, device=None):
    """The call's stream handle. The library launches on the current CUDA
    device, so the call's tensors (on `device`) must live there; with one
    visible device they always do."""
    torch = _torch()
    if device is not None and _device_count() > 1 and device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device} but the current CUDA device is "
                         f"cuda:{torch.cuda.current_device()}: the library launches on the current device")
    if stream is None:
        # the current stream's handle without the Stream object around it (0.1 against 2.8 us)
        index = torch.cuda.current_device() if device is None else device.index
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(index))
    return ctypes.c_void_p(stream.cuda_stream)


def _is_device_tensor(t) -> bool:
    return t.is_cuda


def _ptr(t, dtypes, name, nbytes=0, device=None):
    """Data pointer of `t` after the checks a plain C pointer cannot carry:
    dtype, residency on the call's device, contiguity, and room for the
    `nbytes` bytes the call reads or writes through it."""
    if t is None:
        return None
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not _is_device_tensor(t):
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.nbytes < nbytes:
        raise ValueError(f"{name} holds {t.nbytes} bytes, the call needs {nbytes}")
    return ctypes.c_void_p(t.data_ptr())


_BF16 = None


def _bf16_types():
    global _BF16
    if _BF16 is None:
        torch = _torch()
        _BF16 = (torch.bfloat16, torch.int16, torch.uint16)
    return _BF16


@functools.lru_cache(maxsize=1024)
def _packed_bytes(N: int, K: int, group: int, form: int, gateup: bool) -> int:
    L = lib()
    f = L.w4a16_gateup_repacked_bytes if gateup else L.w4a16_repacked_bytes
    return int(f(N, K, group, form))


def _canonical_bytes(N: int, K: int, group: int):
    """Bytes of a canonical weight's qweight (int32 [N, K/8]), scales or
    biases (bf16 [N, K/G]) and zeros (int32 [N, ceil(K/G/8)])."""
    groups = K // group if group > 0 else 0
    return N * K // 2, N * groups * 2, N * ((groups + 7) // 8) * 4


def _x_rows(x, K) -> int:
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, k = x.shape
    if k != K:
        raise ValueError("x must be [M, K]")
    return M


def repacked_bytes(N: int, K: int, group: int, sym: bool) -> int:
    return int(lib().w4a16_repacked_bytes(N, K, group, int(sym)))


def gateup_repacked_bytes(N_each: int, K: int, group: int, sym: bool) -> int:
    return int(lib().w4a16_gateup_repacked_bytes(N_each, K, group, int(sym)))


def repack(qweight, scales, zeros, N, K, group, sym, stream=None, out=None):
    """Canonical (qweight int32 [N, K/8], scales bf16 [N, K/G], zeros int32) -> packed uint8 tensor."""
    torch = _torch()
    nbytes = repacked_bytes(N, K, group, sym)
    if nbytes == 0:
        raise W4A16Error("repack: unsupported sizes")
    d = qweight.device
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=d)
    bq, bs, bz = _canonical_bytes(N, K, group)
    rc = lib().w4a16_repack(_ptr(qweight, (torch.int32,), "qweight", bq, d),
                            _ptr(scales, _bf16_types(), "scales", bs, d),
                            _ptr(zeros, (torch.int32,), "zeros", bz, d), N, K, group, int(sym),
                            _ptr(out, (torch.uint8,), "out", nbytes, d), _stream(stream, d))
    _check(rc, "w4a16_repack")
    return out


def repack_gateup(qw_gate, sc_gate, z_gate, qw_up, sc_up, z_up, N_each, K, group, sym, stream=None):
    torch = _torch()
    nbytes = gateup_repacked_bytes(N_each, K, group, sym)
    if nbytes == 0:
        raise W4A16Error("repack_gateup: unsupported sizes")
    d = qw_gate.device
    out = torch.empty(nbytes, dtype=torch.uint8, device=d)
    i32, b16 = (torch.int32,), _bf16_types()
    bq, bs, bz = _canonical_bytes(N_each, K, group)
    rc = lib().w4a16_repack_gateup(_ptr(qw_gate, i32, "qw_gate", bq, d), _ptr(sc_gate, b16, "sc_gate", bs, d),
                                   _ptr(z_gate, i32, "z_gate", bz, d), _ptr(qw_up, i32, "qw_up", bq, d),
                                   _ptr(sc_up, b16, "sc_up", bs, d), _ptr(z_up, i32, "z_up", bz, d), N_each, K,
                                   group, int(sym), ctypes.c_void_p(out.data_ptr()), _stream(stream, d))
    _check(rc, "w4a16_repack_gateup")
    return out


def gemm(x, packed, N, K, group, sym, out=None, stream=None):
    """y[M, N] (bf16) = x[M, K] (bf16) . dequant(W)^T."""
    torch = _torch()
    M = _x_rows(x, K)
    d = x.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=d)
    rc = lib().w4a16_gemm(_ptr(x, _bf16_types(), "x", 0, d),
                          _ptr(packed, (torch.uint8,), "packed", _packed_bytes(N, K, group, int(sym), False), d),
                          None, None, M, N, K, group, int(sym), _ptr(out, _bf16_types(), "out", 2 * M * N, d),
                          _stream(stream, d))
    _check(rc, "w4a16_gemm")
    return out


def gemm_argmax(x, packed, N, K, group, sym, out=None, logits=False, stream=None, index_out=None):
    """int64 [M]: the first column of each row of y = x . dequant(W)^T (bf16)
    at which y is largest (torch.argmax over the bf16 row). For M <= 32 the
    logits are stored only when `logits` is true or `out` is given; returns
    (argmax, y or None)."""
    torch = _torch()
    M = _x_rows(x, K)
    d = x.device
    if out is None and (logits or M > 32):
        out = torch.empty((M, N), dtype=torch.bfloat16, device=d)
    idx = index_out if index_out is not None else torch.empty(M, dtype=torch.int64, device=d)
    rc = lib().w4a16_gemm_argmax(_ptr(x, _bf16_types(), "x", 0, d),
                                 _ptr(packed, (torch.uint8,), "packed", _packed_bytes(N, K, group, int(sym), False),
                                      d),
                                 M, N, K, group, int(sym), _ptr(out, _bf16_types(), "out", 2 * M * N, d),
                                 _ptr(idx, (torch.int64,), "index_out", 8 * M, d), _stream(stream, d))
    _check(rc, "w4a16_gemm_argmax")
    return idx, out


TOPK_MAX_K = 1024


def _topk_outs(M, k, d, index_out, values_out, values):
    torch = _torch()
    idx = index_out if index_out is not None else torch.empty((M, k), dtype=torch.int64, device=d)
    vals = values_out
    if vals is None and values:
        vals = torch.empty((M, k), dtype=torch.bfloat16, device=d)
    return idx, vals


def topk(y, k, index_out=None, values_out=None, values=True, stream=None):
    """The k largest entries of every row of the bf16 logits y [M, N], largest
    first (equal values lowest column first, -0 = +0, NaN above +inf).
    Returns (indices int64 [M, k], values bf16 [M, k] or None)."""
    torch = _torch()
    if y.dim() != 2:
        raise ValueError("y must be [M, N]")
    M, N = y.shape
    d = y.device
    idx, vals = _topk_outs(M, k, d, index_out, values_out, values)
    rc = lib().w4a16_topk(_ptr(y, _bf16_types(), "y", 2 * M * N, d), M, N, k,
                          _ptr(idx, (torch.int64,), "index_out", 8 * M * k, d),
                          _ptr(vals, _bf16_types(), "values_out", 2 * M * k, d), _stream(stream, d))
    _check(rc, "w4a16_topk")
    return idx, vals


def gemm_topk(x, packed, N, K, group, sym, k, out=None, index_out=None, values_out=None, values=True, stream=None):
    """y = x . dequant(W)^T (bf16, into `out` or a new tensor), then the top-k
    of each row of y. Returns (indices, values or None, y)."""
    torch = _torch()
    M = _x_rows(x, K)
    d = x.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=d)
    idx, vals = _topk_outs(M, k, d, index_out, values_out, values)
    rc = lib().w4a16_gemm_topk(_ptr(x, _bf16_types(), "x", 0, d),
                               _ptr(packed, (torch.uint8,), "packed", _packed_bytes(N, K, group, int(sym), False), d),
                               M, N, K, group, int(sym), k, _ptr(out, _bf16_types(), "out", 2 * M * N, d),
                               _ptr(idx, (torch.int64,), "index_out", 8 * M * k, d),
                               _ptr(vals, _bf16_types(), "values_out", 2 * M * k, d), _stream(stream, d))
    _check(rc, "w4a16_gemm_topk")
    return idx, vals, out


def gateup_silu(x, packed_gateup, N_each, K, group, sym, out=None, stream=None):
    """h[M, N_each] (bf16) = SiLU(x Wg^T) * (x Wu^T)."""
    torch = _torch()
    M = _x_rows(x, K)
    d = x.device
    if out is None:
        out = torch.empty((M, N_each), dtype=torch.bfloat16, device=d)
    rc = lib().w4a16_gateup_silu(_ptr(x, _bf16_types(), "x", 0, d),
                                 _ptr(packed_gateup, (torch.uint8,), "packed",
                                      _packed_bytes(N_each, K, group, int(sym), True), d),
                                 M, N_each, K, group, int(sym), _ptr(out, _bf16_types(), "out", 2 * M * N_each, d),
                                 _stream(stream, d))
    _check(rc, "w4a16_gateup_silu")
    return out


def repack_affine(qweight, scales, biases, N, K, group, stream=None):
    """Canonical affine weight (qweight int32 [N, K/8], scales and biases bf16 [N, K/G]) -> packed uint8."""
    torch = _torch()
    nbytes = repacked_bytes(N, K, group, AFFINE)
    if nbytes == 0:
        raise W4A16Error("repack_affine: unsupported sizes")
    d = qweight.device
    out = torch.empty(nbytes, dtype=torch.uint8, device=d)
    b16 = _bf16_types()
    bq, bs, _ = _canonical_bytes(N, K, group)
    rc = lib().w4a16_repack_affine(_ptr(qweight, (torch.int32,), "qweight", bq, d),
                                   _ptr(scales, b16, "scales", bs, d), _ptr(biases, b16, "biases", bs, d), N, K,
                                   group, ctypes.c_void_p(out.data_ptr()), _stream(stream, d))
    _check(rc, "w4a16_repack_affine")
    return out


def repack_affine_gateup(qw_gate, sc_gate, b_gate, qw_up, sc_up, b_up, N_each, K, group, stream=None):
    torch = _torch()
    nbytes = gateup_repacked_bytes(N_each, K, group, AFFINE)
    if nbytes == 0:
        raise W4A16Error("repack_affine_gateup: unsupported sizes")
    d = qw_gate.device
    out = torch.empty(nbytes, dtype=torch.uint8, device=d)
    i32, b16 = (torch.int32,), _bf16_types()
    bq, bs, _ = _canonical_bytes(N_each, K, group)
    rc = lib().w4a16_repack_affine_gateup(_ptr(qw_gate, i32, "qw_gate", bq, d), _ptr(sc_gate, b16, "sc_gate", bs, d),
                                          _ptr(b_gate, b16, "b_gate", bs, d), _ptr(qw_up, i32, "qw_up", bq, d),
                                          _ptr(sc_up, b16, "sc_up", bs, d), _ptr(b_up, b16, "b_up", bs, d), N_each,
                                          K, group, ctypes.c_void_p(out.data_ptr()), _stream(stream, d))
    _check(rc, "w4a16_repack_affine_gateup")
    return out


def xsum_bytes(M: int, K: int, group: int) -> int:
    return int(lib().w4a16_xsum_bytes(M, K, group))


def xsum(x, K, group, out=None, stream=None):
    """bf16 [M, kb3]: the sum of x[m] over each group g as three bf16 parts
    (hi, mid, lo at columns 3g .. 3g+2) that add up to the float32 sum exactly."""
    torch = _torch()
    M = _x_rows(x, K)
    nbytes = xsum_bytes(M, K, group)
    if nbytes == 0:
        raise W4A16Error("xsum: unsupported sizes")
    d = x.device
    if out is None:
        out = torch.empty((M, nbytes // 2 // M), dtype=torch.bfloat16, device=d)
    rc = lib().w4a16_xsum(_ptr(x, _bf16_types(), "x", 0, d), M, K, group,
                          _ptr(out, _bf16_types(), "out", nbytes, d), _stream(stream, d))
    _check(rc, "w4a16_xsum")
    return out


def _xs_ptr(xs, M, K, group, d):
    # the table is read only by the tcgen05 GEMM (M > 32), but whenever one is
    # passed it must be whole
    return None if xs is None else _ptr(xs, _bf16_types(), "xsum", xsum_bytes(M, K, group), d)


def gemm_affine(x, packed, N, K, group, xs=None, out=None, stream=None):
    """y[M, N] (bf16) = x . (scale * q + bias)^T. `xs` (from xsum) is needed
    for M > 32; None lets the M <= 32 kernels form the group sums themselves."""
    torch = _torch()
    M = _x_rows(x, K)
    d = x.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=d)
    rc = lib().w4a16_gemm_affine(_ptr(x, _bf16_types(), "x", 0, d), _xs_ptr(xs, M, K, group, d),
                                 _ptr(packed, (torch.uint8,), "packed", _packed_bytes(N, K, group, AFFINE, False), d),
                                 M, N, K, group, _ptr(out, _bf16_types(), "out", 2 * M * N, d), _stream(stream, d))
    _check(rc, "w4a16_gemm_affine")
    return out


def gemm_affine_noalloc(x, packed, N, K, group, out=None, stream=None):
    """gemm_affine with the group sums in the library's fixed device array (no
    table argument; calls in flight at once on one device race on it)."""
    torch = _torch()
    M = _x_rows(x, K)
    d = x.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=d)
    rc = lib().w4a16_gemm_affine_noalloc(_ptr(x, _bf16_types(), "x", 0, d),
                                         _ptr(packed, (torch.uint8,), "packed",
                                              _packed_bytes(N, K, group, AFFINE, False), d),
                                         M, N, K, group, _ptr(out, _bf16_types(), "out", 2 * M * N, d),
                                         _stream(stream, d))
    _check(rc, "w4a16_gemm_affine_noalloc")
    return out


def affine_bits_repacked_bytes(N: int, K: int, group: int, bits: int) -> int:
    return int(lib().w4a16_affine_bits_repacked_bytes(N, K, group, bits))


def affine_bits_scratch_bytes(M: int, K: int, group: int, bits: int) -> int:
    return int(lib().w4a16_affine_bits_scratch_bytes(M, K, group, bits))


def repack_affine_bits(qweight, scales, biases, N, K, group, bits, stream=None):
    """Canonical b-bit affine weight (qweight uint32/int32 [N, ceil(K*bits/32)],
    one bit stream per row; scales and biases bf16 [N, K/G]) -> packed uint8."""
    torch = _torch()
    nbytes = affine_bits_repacked_bytes(N, K, group, bits)
    if nbytes == 0:
        raise W4A16Error(f"unsupported b-bit affine weight N={N} K={K} group={group} bits={bits}")
    d = qweight.device
    out = torch.empty(nbytes, dtype=torch.uint8, device=d)
    qbytes = N * ((K * bits + 31) // 32) * 4
    _, sbytes, _ = _canonical_bytes(N, K, group)
    rc = lib().w4a16_repack_affine_bits(_ptr(qweight, (torch.int32, torch.uint32), "qweight", qbytes, d),
                                        _ptr(scales, _bf16_types(), "scales", sbytes, d),
                                        _ptr(biases, _bf16_types(), "biases", sbytes, d), N, K, group, bits,
                                        _ptr(out, (torch.uint8,), "packed", nbytes, d), _stream(stream, d))
    _check(rc, "w4a16_repack_affine_bits")
    return out


def gemm_affine_bits(x, packed, N, K, group, bits, scratch=None, out=None, stream=None):
    """y[M, N] (bf16) = x . (scale * q + bias)^T of a b-bit affine weight;
    `scratch` (uint8, affine_bits_scratch_bytes) is allocated when not given."""
    torch = _torch()
    M = _x_rows(x, K)
    d = x.device
    sbytes = affine_bits_scratch_bytes(M, K, group, bits)
    if sbytes == 0:
        raise W4A16Error(f"unsupported b-bit affine call M={M} K={K} group={group} bits={bits}")
    if scratch is None:
        scratch = torch.empty(sbytes, dtype=torch.uint8, device=d)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=d)
    rc = lib().w4a16_gemm_affine_bits(_ptr(x, _bf16_types(), "x", 2 * M * K, d),
                                      _ptr(scratch, (torch.uint8,), "scratch", sbytes, d),
                                      _ptr(packed, (torch.uint8,), "packed", affine_bits_repacked_bytes(N, K, group, bits),
                                           d),
                                      M, N, K, group, bits, _ptr(out, _bf16_types(), "out", 2 * M * N, d),
                                      _stream(stream, d))
    _check(rc, "w4a16_gemm_affine_bits")
    return out


def dequantize_affine_bits(packed, N, K, group, bits, stream=None):
    """float32 [N, K]: scale * q + bias read back from a b-bit packed weight."""
    torch = _torch()
    d = packed.device
    w = torch.empty((N, K), dtype=torch.float32, device=d)
    rc = lib().w4a16_dequantize_affine_bits(_ptr(packed, (torch.uint8,), "packed",
                                                 affine_bits_repacked_bytes(N, K, group, bits), d),
                                            N, K, group, bits, _ptr(w, (torch.float32,), "w_out", 4 * N * K, d),
                                            _stream(stream, d))
    _check(rc, "w4a16_dequantize_affine_bits")
    return w


def gateup_silu_affine(x, packed_gateup, N_each, K, group, xs=None, out=None, stream=None):
    """h[M, N_each] (bf16) = SiLU(x Wg^T) * (x Wu^T), affine weights."""
    torch = _torch()
    M = _x_rows(x, K)
    d = x.device
    if out is None:
        out = torch.empty((M, N_each), dtype=torch.bfloat16, device=d)
    rc = lib().w4a16_gateup_silu_affine(_ptr(x, _bf16_types(), "x", 0, d), _xs_ptr(xs, M, K, group, d),
                                        _ptr(packed_gateup, (torch.uint8,), "packed",
                                             _packed_bytes(N_each, K, group, AFFINE, True), d),
                                        M, N_each, K, group, _ptr(out, _bf16_types(), "out", 2 * M * N_each, d),
                                        _stream(stream, d))
    _check(rc, "w4a16_gateup_silu_affine")
    return out


def dequantize(packed, N, K, group, sym, stream=None):
    """float32 [N, K] = (q - z) * scale (exact), or scale * q + bias rounded once
    to float32 for sym = AFFINE, read back through the kernels' unpack."""
    torch = _torch()
    d = packed.device
    need = _packed_bytes(N, K, group, int(sym), False)
    p = _ptr(packed, (torch.uint8,), "packed", need, d)
    out = torch.empty((N, K), dtype=torch.float32, device=d)
    rc = lib().w4a16_dequantize(p, N, K, group, int(sym), ctypes.c_void_p(out.data_ptr()), _stream(stream, d))
    _check(rc, "w4a16_dequantize")
    return out


# ---------------------------------------------------------------------------
# Paged key/value cache and the attention of drafted token trees. A call with
# nothing to do (no rows, no new tokens, no rows named) checks its arguments,
# launches nothing, and its outputs say so.
# ---------------------------------------------------------------------------
MAX_TREE = 64     # new tokens of a sequence in one attention or acceptance call
MAX_ROWS = 4096   # rows that one fork, free or reserve call may name

# w4a16_kv_cache: k, v, k_scale, v_scale; layer, page, head and row strides of
# each; layers, pages, kv_heads, page_rows, dim, type
_KV_BASES = _struct.Struct("=4Q")
_KV_SHAPE = _struct.Struct("=8q6i")


class _Types:
    """torch's dtypes, looked up once (the module loads without torch)."""
    def __init__(self):
        torch = _torch()
        self.bf16, self.e4m3, self.i32, self.i64 = torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.int64
        self.f32, self.u8, self.empty = torch.float32, torch.uint8, torch.empty


_types = functools.lru_cache(maxsize=1)(_Types)


# These calls are short on the device, so their checks are written for speed:
# get_device() (an int) stands for the device, and a message is only put
# together once something is wrong.
def _refuse(t, dtype, name, dev, need=None):
    """Raise what is wrong with tensor `t`: its type, place, order or size."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype} is not {dtype}")
    if not _is_device_tensor(t):
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on device {dev}")
    if need is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if need is not None:
        raise ValueError(f"{name} has shape {list(t.shape)}, the call needs {need} elements")


def _flat(t, dtype, name, need, dev):
    """Data pointer of a contiguous tensor of exactly `need` elements."""
    if t.dtype is not dtype or t.get_device() != dev or t.numel() != need or not t.is_contiguous():
        _refuse(t, dtype, name, dev, need)
    return t.data_ptr()


def _table(t, dev):
    """Data pointer, rows and width of an int32 page table."""
    if t.dtype is not _types().i32 or t.get_device() != dev or t.dim() != 2 or not t.is_contiguous():
        _refuse(t, _types().i32, "page_table", dev, "[rows, max pages] int32")
    rows, width = t.shape
    return t.data_ptr(), rows, width


def _place(t, name):
    """The device number of the tensor that names the call's device."""
    dev = t.get_device()
    if dev < 0 and not _is_device_tensor(t):
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _on(stream, t):
    """The call's stream handle, as _stream gives it."""
    return _stream(stream, t.device)


def _empty(shape, dtype, like, stream):
    """A new tensor on `like`'s device, taken from the pool of the stream that
    will write it (so that nothing still running elsewhere uses its memory)."""
    if stream is None:
        return _types().empty(shape, dtype=dtype, device=like.device)
    with _torch().cuda.stream(stream):
        return _types().empty(shape, dtype=dtype, device=like.device)


def _capturing(stream):
    """Whether the call's stream (the current one if None) is being captured."""
    cuda = _torch().cuda
    if stream is None:
        return cuda.is_current_stream_capturing()
    with cuda.stream(stream):
        return cuda.is_current_stream_capturing()


_small_outputs = {}
_SMALL, _AT_ONCE = 16384, 32  # bytes of a small output, how many are made at once


def _small_out(shape, dtype, like, dev, stream, handle):
    """A new tensor, as _empty gives it. Small ones are made 32 at a time, out
    of one allocation: on their own three of them cost more than the call that
    fills them (10 us against 6; a 10 KB output, mean of many calls on the host:
    17.7 us on its own, 15.6 so, one call in 32 taking 50). Each is handed out once, as a plain
    tensor (no view and with a version counter of its own: unsafe_split's, not
    unbind's; not an inference tensor, whatever mode the batch is made in);
    their common memory goes back to the stream's pool with the last of them.
    Under capture every output comes from the graph's pool."""
    torch = _torch()
    if _capturing(stream):
        return _empty(shape, dtype, like, stream)
    key = (shape, dtype, dev, handle)
    try:
        return _small_outputs[key].pop()  # (one step, whatever other threads do)
    except (KeyError, IndexError):
        pass
    n = dtype.itemsize
    for d in shape:
        n *= d
    if n > _SMALL or n == 0:
        return _empty(shape, dtype, like, stream)
    if torch.is_inference_mode_enabled():
        with torch.inference_mode(False):
            return _small_out(shape, dtype, like, dev, stream, handle)
    batch = _empty((_AT_ONCE * shape[0], *shape[1:]), dtype, like, stream)
    ready = list(batch.unsafe_split(shape[0]))
    out = ready.pop()
    if len(_small_outputs) >= 256:
        _small_outputs.clear()
    _small_outputs[key] = ready
    return out


_workspaces = {}
_KEPT = 8  # workspaces kept, of the streams that began to use one last
# Held while a call takes the kept workspace and makes its launches: there are
# two, and another host thread's on the same stream must not come between them.
_kept_workspace = _threading.RLock()


def _workspace(need, like, dev, stream, handle):
    """The scratch of calls that bring none: one buffer per device and stream,
    used by one call after the other in the stream's order (the caller holds
    _kept_workspace), and grown when a call needs more. A call under capture
    gets a buffer of its own from the graph's pool, which lives as long as the
    graph."""
    if _capturing(stream):
        return _empty(need, _types().u8, like, stream)
    key = (dev, handle)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = _workspaces[key] = _empty(need, _types().u8, like, stream)
        while len(_workspaces) > _KEPT:  # goes back to its stream's pool, behind the calls that use it
            del _workspaces[next(iter(_workspaces))]
    return ws


@functools.lru_cache(maxsize=1024)
def _kv_shape(shape, ks, vs, e4m3):
    """The part of w4a16_kv_cache that shape and strides make (the same for all layers of a model)."""
    if ks[-1] != 1 or vs[-1] != 1:
        raise ValueError("k_cache, v_cache: the last axis must be contiguous")
    if len(ks) == 4:
        ks, vs = (0, *ks), (0, *vs)
    return _KV_SHAPE.pack(*ks[:4], *vs[:4], *shape, e4m3)


def _kv_cache(k_cache, v_cache, k_scale, v_scale, one_layer, dev):
    """The w4a16_kv_cache bytes of a cache given as [pages, kv heads, page
    rows, dim] tensors (any strides, dim contiguous), or with a leading layer
    axis unless `one_layer`; and its shape with that axis."""
    ty = _types()
    shape = k_cache.shape
    axes = len(shape)
    if axes != 4 and (one_layer or axes != 5):
        raise ValueError("k_cache must be [pages, kv heads, page rows, dim]" +
                         ("" if one_layer else ", or that with a leading layer axis"))
    if v_cache.shape != shape:
        raise ValueError(f"v_cache has shape {list(v_cache.shape)}, k_cache {list(shape)}")
    dt = k_cache.dtype
    e4m3 = dt is ty.e4m3
    if (not e4m3 and dt is not ty.bf16) or v_cache.dtype is not dt:
        raise TypeError(f"k_cache, v_cache: dtypes {dt}, {v_cache.dtype} are not both bfloat16 or both float8_e4m3fn")
    if k_cache.get_device() != dev:
        _refuse(k_cache, dt, "k_cache", dev)
    if v_cache.get_device() != dev:
        _refuse(v_cache, dt, "v_cache", dev)
    if axes == 4:
        shape = (1, *shape)
    tail = _kv_shape(shape, k_cache.stride(), v_cache.stride(), e4m3)
    kp = vp = 0
    if e4m3 and one_layer:
        if k_scale is None or v_scale is None:
            raise ValueError("a float8_e4m3fn cache needs k_scale and v_scale")
        kp = _flat(k_scale, ty.f32, "k_scale", shape[2], dev)
        vp = _flat(v_scale, ty.f32, "v_scale", shape[2], dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to float8_e4m3fn caches")
    return _KV_BASES.pack(k_cache.data_ptr(), v_cache.data_ptr(), kp, vp) + tail, shape


def _token_rows(t, name, dim, dev):
    """Pointer, strides and sizes of a bf16 [tokens, heads, dim] tensor whose last axis is contiguous."""
    if t.dtype is not _types().bf16 or t.get_device() != dev:
        _refuse(t, _types().bf16, name, dev)
    shape, s = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, heads, {dim}], not {list(shape)}")
    if s[2] != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return t.data_ptr(), s[0], s[1], shape[0], shape[1]


def _fill(t, value, stream):
    """`value` throughout an output of a call that has nothing to launch."""
    if stream is None:
        return t.fill_(value)
    with _torch().cuda.stream(stream):
        return t.fill_(value)


def kv_append(k, v, k_cache, v_cache, page_table, lengths, starts, k_scale=None, v_scale=None, stream=None):
    """Write the new tokens' keys and values (bf16 [tokens, kv heads, dim],
    strided views allowed) behind each row's context: token starts[b] + i goes
    to position lengths[b] + i of row b. page_table int32 [rows, max pages],
    lengths int32 [rows], starts int32 [rows + 1]. e4m3 caches store x /
    scale[head], rounded to nearest and saturated."""
    ty, dev = _types(), _place(k, "k")
    cache, (_, _, heads, _, dim) = _kv_cache(k_cache, v_cache, k_scale, v_scale, True, dev)
    kp, kt, kh, tokens, k_heads = _token_rows(k, "k", dim, dev)
    vp, vt, vh, v_tokens, v_heads = _token_rows(v, "v", dim, dev)
    if v_tokens != tokens or k_heads != heads or v_heads != heads:
        raise ValueError(f"k and v must both be [tokens, {heads}, {dim}], not {list(k.shape)} and {list(v.shape)}")
    table, rows, width = _table(page_table, dev)
    lengths, starts = _flat(lengths, ty.i32, "lengths", rows, dev), _flat(starts, ty.i32, "starts", rows + 1, dev)
    if rows == 0 or tokens == 0:
        return
    rc = lib().w4a16_kv_append(kp, vp, kt, kh, vt, vh, cache, table, width, lengths, starts, rows, tokens, _on(stream, k))
    _check(rc, "w4a16_kv_append")


@functools.lru_cache(maxsize=1024)
def tree_attention_workspace_bytes(heads: int, kv_heads: int, dim: int, max_tree: int) -> int:
    return int(lib().w4a16_tree_attention_workspace_bytes(heads, kv_heads, dim, max_tree))


def tree_attention(q, k_cache, v_cache, page_table, lengths, starts, mask, max_tree, scale=None, k_scale=None,
                   v_scale=None, out=None, workspace=None, stream=None):
    """bf16 [tokens, heads, dim]: attention of the new tokens over their rows'
    paged contexts and, as the int64 [tokens] mask words say (bit j: new token
    j of the row; None: a causal chain), over one another. q bf16 [tokens,
    heads, dim] (strided views allowed); every row has at most max_tree <=
    MAX_TREE new tokens, appended before. scale defaults to dim ** -0.5. A token
    that sees nothing gets 0; padding tokens (at starts[rows] and above) are
    left as they are in `out`. Without a `workspace` (uint8,
    tree_attention_workspace_bytes) the call uses one that the module keeps
    for its stream; a given one belongs to one call at a time (host threads
    that share a stream need one each)."""
    ty, dev = _types(), _place(q, "q")
    cache, (_, _, kv_heads, _, dim) = _kv_cache(k_cache, v_cache, k_scale, v_scale, True, dev)
    qp, qt, qh, tokens, heads = _token_rows(q, "q", dim, dev)
    need = tree_attention_workspace_bytes(heads, kv_heads, dim, max_tree)
    if need == 0:
        raise W4A16Error(f"tree_attention: unsupported heads={heads} kv_heads={kv_heads} dim={dim} max_tree={max_tree}")
    table, rows, width = _table(page_table, dev)
    handle = _on(stream, q)
    if workspace is not None and (workspace.dtype is not ty.u8 or workspace.get_device() != dev or not workspace.is_contiguous() or workspace.numel() < need):
        _refuse(workspace, ty.u8, "workspace", dev, need)
    if out is None:
        # (the sizes of one or two tokens; a larger call is longer on the device than here)
        if 2 * tokens * heads * dim <= _SMALL:
            out = _small_out((tokens, heads, dim), ty.bf16, q, dev, stream, handle.value)
        else:
            out = _empty((tokens, heads, dim), ty.bf16, q, stream)
    args = (qp, qt, qh, cache, table, width, _flat(lengths, ty.i32, "lengths", rows, dev),
            _flat(starts, ty.i32, "starts", rows + 1, dev), None if mask is None else _flat(mask, ty.i64, "mask", tokens, dev),
            rows, tokens, heads, max_tree, dim ** -0.5 if scale is None else scale,
            _flat(out, ty.bf16, "out", tokens * heads * dim, dev))
    if rows == 0 or tokens == 0:
        return out
    call = lib().w4a16_tree_attention
    if workspace is not None:
        rc = call(*args, workspace.data_ptr(), handle)
    else:
        with _kept_workspace:
            rc = call(*args, _workspace(need, q, dev, stream, handle.value).data_ptr(), handle)
    _check(rc, "w4a16_tree_attention")
    return out


def tree_accept(target, draft, mask, starts, max_tree, path=None, count=None, token=None, stream=None):
    """Greedy walk down each row's draft tree: target int64 [tokens] the
    model's pick after each node (gemm_argmax), draft int64 [tokens] the drafted
    tokens, mask as in tree_attention. Returns (path int32 [rows, max_tree]:
    the accepted nodes, then -1; count int32 [rows]; token int64 [rows]: the
    pick after the last accepted node)."""
    ty, dev = _types(), _place(target, "target")
    tokens, rows = target.numel(), starts.numel() - 1
    handle = _on(stream, target)
    if path is None:
        path = _small_out((rows, max_tree), ty.i32, target, dev, stream, handle.value)
    if count is None:
        count = _small_out((rows,), ty.i32, target, dev, stream, handle.value)
    if token is None:
        token = _small_out((rows,), ty.i64, target, dev, stream, handle.value)
    args = (_flat(target, ty.i64, "target", tokens, dev), _flat(draft, ty.i64, "draft", tokens, dev),
            None if mask is None else _flat(mask, ty.i64, "mask", tokens, dev),
            _flat(starts, ty.i32, "starts", rows + 1, dev), rows, tokens, max_tree,
            _flat(path, ty.i32, "path", rows * max_tree, dev), _flat(count, ty.i32, "count", rows, dev),
            _flat(token, ty.i64, "token", rows, dev), handle)
    if rows == 0 or tokens == 0:
        _check(0 if 1 <= max_tree <= MAX_TREE else -1, "w4a16_tree_accept")
        return _fill(path, -1, stream), _fill(count, 0, stream), _fill(token, -1, stream)
    _check(lib().w4a16_tree_accept(*args), "w4a16_tree_accept")
    return path, count, token


def kv_compact(k_cache, v_cache, page_table, lengths, path, count, lengths_out=None, stream=None):
    """Move the accepted rows together in every layer of the cache ([layers,]
    pages, kv heads, page rows, dim): position lengths[b] + path[b, i] to
    lengths[b] + i for i < count[b]. Returns the new lengths, lengths + count
    (a new tensor, or `lengths_out`, which must not be `lengths`)."""
    ty, dev = _types(), _place(k_cache, "k_cache")
    cache, _ = _kv_cache(k_cache, v_cache, None, None, False, dev)
    table, rows, width = _table(page_table, dev)
    if path.dim() != 2:
        raise ValueError(f"path must be [{rows}, max_tree], not {list(path.shape)}")
    max_tree = path.shape[1]
    handle = _on(stream, k_cache)
    if lengths_out is None:
        lengths_out = _small_out((rows,), ty.i32, k_cache, dev, stream, handle.value)
    args = (cache, table, width, _flat(lengths, ty.i32, "lengths", rows, dev),
            _flat(path, ty.i32, "path", rows * max_tree, dev), _flat(count, ty.i32, "count", rows, dev), rows, max_tree,
            _flat(lengths_out, ty.i32, "lengths_out", rows, dev), handle)
    if rows:
        _check(lib().w4a16_kv_compact(*args), "w4a16_kv_compact")
    return lengths_out


def kv_free(page_table, lengths, refs, rows, stream=None):
    """Drop the table rows `rows` (int32 [n], distinct): one reference (refs
    int32 [pages]) of each page they hold; their entries become -1, their
    lengths 0."""
    i32, dev = _types().i32, _place(page_table, "page_table")
    table, table_rows, width = _table(page_table, dev)
    pages, n = refs.numel(), rows.numel()
    args = (table, width, table_rows, _flat(lengths, i32, "lengths", table_rows, dev), _flat(refs, i32, "refs", pages, dev),
            pages, _flat(rows, i32, "rows", n, dev), n, _on(stream, page_table))
    if n:
        _check(lib().w4a16_kv_free(*args), "w4a16_kv_free")


def kv_fork(k_cache, v_cache, page_table, lengths, refs, src, dst, ok=None, stream=None):
    """Branch: the empty table row dst[j] becomes a copy of row src[j] (int32
    [n]). Whole pages are shared, a part-filled last page is copied in every
    layer into the lowest free page. Returns ok int32 [1]: 1, or 0 when the
    free pages did not suffice and nothing changed."""
    ty, dev = _types(), _place(page_table, "page_table")
    i32 = ty.i32
    cache, shape = _kv_cache(k_cache, v_cache, None, None, False, dev)
    table, table_rows, width = _table(page_table, dev)
    handle = _on(stream, page_table)
    if ok is None:
        ok = _small_out((1,), i32, page_table, dev, stream, handle.value)
    n = src.numel()
    args = (cache, table, width, table_rows, _flat(lengths, i32, "lengths", table_rows, dev),
            _flat(refs, i32, "refs", shape[1], dev), _flat(src, i32, "src", n, dev), _flat(dst, i32, "dst", n, dev), n,
            _flat(ok, i32, "ok", 1, dev), handle)
    if n == 0:
        return _fill(ok, 1, stream)
    _check(lib().w4a16_kv_fork(*args), "w4a16_kv_fork")
    return ok


def kv_reserve(page_table, refs, rows, want, page_rows, ok=None, stream=None):
    """Room to grow: table row rows[j] gets the lowest free pages until it
    holds want[j] tokens (int32 [n] each). Returns ok int32 [1]: 1, or 0 when
    the free pages did not suffice and nothing changed."""
    ty, dev = _types(), _place(page_table, "page_table")
    i32 = ty.i32
    table, table_rows, width = _table(page_table, dev)
    handle = _on(stream, page_table)
    if ok is None:
        ok = _small_out((1,), i32, page_table, dev, stream, handle.value)
    n, pages = rows.numel(), refs.numel()
    args = (table, width, table_rows, _flat(refs, i32, "refs", pages, dev), pages, page_rows,
            _flat(rows, i32, "rows", n, dev), _flat(want, i32, "want", n, dev), n, _flat(ok, i32, "ok", 1, dev), handle)
    if n == 0:
        _check(0 if page_rows in (16, 32, 64, 128, 256) else -1, "w4a16_kv_reserve")
        return _fill(ok, 1, stream)
    _check(lib().w4a16_kv_reserve(*args), "w4a16_kv_reserve")
    return ok


def kernel_status() -> int:
    """Synchronise and return (and clear) the kernels' status: 0, -5 (a bounded
    wait gave up) or -6 (a cache call skipped an index outside its buffers)."""
    return int(lib().w4a16_kernel_status())


def set_kernel_override(which: int) -> int:
    return int(lib().w4a16_set_kernel_override(which))


def set_programmatic_overlap(on: bool) -> bool:
    """Let each M <= 32 call start streaming its weights while the previous
    kernel on the stream finishes (x and y are touched only after it has).
    Only while packed weights are read-only and complete; returns the previous
    setting."""
    prev = int(lib().w4a16_set_programmatic_overlap(int(bool(on))))
    if prev < 0:
        raise W4A16Error("w4a16_set_programmatic_overlap: bad value")
    return bool(prev)
