"""ctypes binding of libfa_gb300 (argument marshalling only).

Every function here checks tensor dtypes/devices/shapes, takes raw device
pointers and the current CUDA stream from PyTorch, and calls the C entry
point of the same name.  All compute happens in the CUDA kernels behind the
C ABI; there is no other path.  If the library is not built, loading fails
with an error instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libfa_gb300.so")
TORCH_LIB_PATH = os.path.join(_PKG, "lib", "_fa_torch.so")

FA_OK = 0
STATUS_NAMES = {
    0: "FA_OK", 1: "FA_ERR_NULL", 2: "FA_ERR_ALIGN", 3: "FA_ERR_HEAD_DIM", 4: "FA_ERR_SHAPE",
    5: "FA_ERR_ARCH", 6: "FA_ERR_CUDA", 7: "FA_ERR_TIMEOUT", 8: "FA_ERR_WORKSPACE", 9: "FA_ERR_SCALE",
    10: "FA_ERR_NOT_DEVICE", 11: "FA_ERR_SCRATCH_LIMIT",
    12: "FA_ERR_PAGE",
}

# Exported symbols and their C signatures (include/fa.h).
_P, _I, _F, _Z, _U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint64
_L = ctypes.c_longlong
SIGNATURES = {
    "fa_status_string": (ctypes.c_char_p, [_I]),
    "fa_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P]),
    "fa_bwd_workspace_bytes": (_Z, [_I, _I, _I, _I]),
    "fa_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _I, _I, _I, _I, _F, _I, _P]),
    "fa_fwd_varlen": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_bwd_varlen_workspace_bytes": (_Z, [_I, _I, _I, _I, _I]),
    "fa_bwd_varlen": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_get_device_error": (_I, [_P]),
    "fa_selftest_wait_timeout": (_I, [_U64, _P]),
    "fa_set_kernel_events": (_I, [_P, _P]),
    "fa_cta_order": (_I, [_I, _I, _I, ctypes.POINTER(_I), _P, _P, ctypes.c_longlong]),
    "fa_last_error_detail": (ctypes.c_char_p, []),
    "fa_bwd_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P]),
    "fa_microbench": (_I, [_I, _I, ctypes.POINTER(ctypes.c_double), _P]),
    "fa_fwd_grouped": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _L, _L, _L, _F, _I, _I, _P]),
    "fa_bwd_grouped_workspace_bytes": (_Z, [_I, _I, _I, _I, _I, _I, _I]),
    "fa_bwd_grouped": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P, _I, _I, _I, _I, _I, _I, _L, _L, _L, _F, _I,
                            _I, _P]),
    "fa_cache8_store": (_I, [_P] * 9 + [_I] * 8 + [_L, _L, _P]),
    "fa_decode_cache8_workspace_bytes": (_Z, [_I] * 6),
    "fa_fwd_decode_cache8": (_I, [_P] * 10 + [_Z] + [_I] * 9 + [_F, _I, _P]),
    "fa_rotary": (_I, [_P] * 7 + [_I] * 8 + [_L, _L, _P]),
    "fa_cache8_store_rotary": (_I, [_P] * 14 + [_I] * 12 + [_L, _L, _L, _I, _P]),
    "fa_chunk_cache8_workspace_bytes": (_Z, [_I] * 7),
    "fa_fwd_chunk_cache8": (_I, [_P] * 11 + [_Z] + [_I] * 10 + [_L, _F, _I, _I, _P]),
    "fa_decode_workspace_bytes": (_Z, [_I, _I, _I, _I, _I]),
    "fa_fwd_decode": (_I, [_P, _P, _P, _P, _P, _P, _Z, _I, _I, _I, _I, _I, _F, _I, _P]),
}

# fa_microbench selectors: rate per SM per SM-clock of each unit (the
# MUFU-vs-tensor measurements), and the accuracy of the polynomial exp2.
MICROBENCH = {"ex2_per_sm_clk": 0, "cvt_bf16x2_per_sm_clk": 1, "ffma_per_sm_clk": 2,
              "mma_bf16_flop_per_sm_clk_n256": 3, "mma_bf16_flop_per_sm_clk_n128": 4,
              "mma_bf16_flop_per_sm_clk_n128_tmem_a": 5, "mma_bf16_flop_per_sm_clk_n256_random": 6,
              "mma_bf16_flop_per_sm_clk_n128_tmem_a_random": 7,
              "fwd_mma_stream_flop_per_sm_clk_d128": 8, "fwd_mma_stream_flop_per_sm_clk_pv64": 9,
              "fwd_mma_stream_flop_per_sm_clk_pv64_separate_p": 10,
              "fwd_mma_stream_flop_per_sm_clk_d128_pv_first": 11,
              "softmax_ex2_cvt_per_sm_clk": 38, "softmax_step_per_sm_clk": 40,
              "ex2_poly_max_rel_err": 42, "softmax_step_quarter_poly_per_sm_clk": 43}

# Size of the static scratch array behind fa_bwd_noalloc (FA_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 32 << 20

_lib = None
_native = None
_lock = threading.Lock()


class FaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = f"{fn} failed: {STATUS_NAMES.get(status, status)} ({lib().fa_status_string(status).decode()})"
        if status == 6:
            msg += f": {lib().fa_last_error_detail().decode()}"
        super().__init__(msg)


def lib() -> ctypes.CDLL:
    """Load libfa_gb300.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"{LIB_PATH} is missing: build it with `python -m io_aware_attention_flash_gb300.build`")
                handle = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in SIGNATURES.items():
                    fn = getattr(handle, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = handle
    return _lib


class _NoNative:
    """Stands for the compiled calls where they cannot be loaded: hands every call
    to the helper's Python path, which launches the same kernels."""

    @staticmethod
    def _none(*args):
        return None

    forward_grouped = backward_grouped = flash_attention_grouped = cache8_store = decode_cache8 = _none
    rotary = rotary_embedding = cache8_store_rotary = chunk_cache8 = _none


def native():
    """The compiled calls of the grouped-head and cache entry points (once
    loaded).  Each does what the Python helper of its name does and returns
    None where anything is not in order; the helper then takes the Python path,
    which says what.  Where they are not built, or for another PyTorch, the
    Python paths take every call (and more host time: a warning says so).  Raises
    if libfa_gb300.so has not been built."""
    global _native
    if _native is None:
        lib()
        with _lock:
            if _native is None:
                from . import build

                rebuild = ("calls take more host time until it is rebuilt with "
                           "`python -m io_aware_attention_flash_gb300.build`")
                if not os.path.exists(TORCH_LIB_PATH):
                    warnings.warn(f"{TORCH_LIB_PATH} is missing: {rebuild}", RuntimeWarning, stacklevel=3)
                    _native = _NoNative()
                    return _native
                if build.torch_built_for() != build.torch_stamp():
                    warnings.warn(f"{TORCH_LIB_PATH} was built for another PyTorch or Python "
                                  f"({build.torch_built_for() or 'unknown'}; here {build.torch_stamp()}): {rebuild}",
                                  RuntimeWarning, stacklevel=3)
                    _native = _NoNative()
                    return _native
                spec = importlib.util.spec_from_file_location("_fa_torch", TORCH_LIB_PATH)
                module = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(module)
                _native = module
    return _native


def _check(fn: str, status: int) -> None:
    if status != FA_OK:
        raise FaError(fn, status)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _bf16(name: str, t: torch.Tensor, shape) -> None:
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16 (got {t.dtype}); fp32 and other types are not supported")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _f32(name: str, t: torch.Tensor, shape) -> None:
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous CUDA float32 tensor of shape {tuple(shape)}")


def _scale(scale, d):
    return float(d) ** -0.5 if scale is None else float(scale)


# The checks of the entry points below run on every call of a decoding step, so
# each is one expression where all is well; what is wrong is found out after.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream_of(stream, dev: int) -> int:
    """The given stream, or the current one of the tensors' device."""
    if stream is None:
        return _raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream belongs to cuda:{stream.device_index}, the tensors are on cuda:{dev}")
    return stream.cuda_stream


def _device_of(name: str, t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    return dev


def _dense(name: str, t: torch.Tensor, dtype, shape, dev: int) -> None:
    """Checks a contiguous tensor of the given type and shape on device dev."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return
    if t.dtype is not dtype and dtype in (torch.bfloat16, torch.float8_e4m3fn):
        raise TypeError(f"{name} must be {str(dtype)[6:]} (got {t.dtype}); other types are not supported")
    raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} tensor of shape {tuple(shape)} on cuda:{dev} (got "
                     f"{t.dtype}, {tuple(t.shape)}, strides {t.stride()}, {t.device})")


def _rows(name: str, t: torch.Tensor, rows: int, heads: int, d: int, dev: int) -> int:
    """Checks a bf16 [rows, heads, d] tensor whose rows may be further apart
    than heads·d elements (a slice of a wider projection); returns the row
    stride in elements."""
    n = heads * d
    if t.dtype is torch.bfloat16 and t.get_device() == dev and t.shape == (rows, heads, d):
        if t.is_contiguous() or rows <= 1 and t[0].is_contiguous():
            return n
        s0, s1, s2 = t.stride()
        if s2 == 1 and (s1 == d or heads == 1) and s0 >= n and s0 % 8 == 0:
            return s0
        raise ValueError(f"{name}: each row of {heads} heads of {d} must be contiguous, and rows a multiple of 8 "
                         f"elements and at least {n} apart (strides {t.stride()})")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16 (got {t.dtype}); fp32 and other types are not supported")
    raise ValueError(f"{name} must be a tensor of shape {(rows, heads, d)} on cuda:{dev} (got {tuple(t.shape)}, {t.device})")


def _nbytes(workspace: torch.Tensor, dev: int) -> int:
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def fa_fwd(q, k, v, o, lse, causal: bool, scale=None, stream=None) -> None:
    B, N, H, d = q.shape
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _bf16(n, t, (B, N, H, d))
    _f32("lse", lse, (B, H, N))
    _check("fa_fwd", lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                                  _scale(scale, d), int(bool(causal)), _stream(stream)))


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, H, N, d))


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal: bool, scale=None, stream=None) -> None:
    B, N, H, d = q.shape
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv)):
        _bf16(n, t, (B, N, H, d))
    _f32("lse", lse, (B, H, N))
    _check("fa_bwd", lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                                  _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  B, H, N, d, _scale(scale, d), int(bool(causal)), _stream(stream)))


def fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, causal: bool, scale=None, stream=None) -> None:
    """fa_bwd for callers that cannot provide device memory: the library's
    static scratch array stands in for the workspace (problems up to
    NOALLOC_SCRATCH_BYTES of workspace; calls must not overlap on the GPU)."""
    B, N, H, d = q.shape
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv)):
        _bf16(n, t, (B, N, H, d))
    _f32("lse", lse, (B, H, N))
    _check("fa_bwd_noalloc", lib().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                                  _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, _scale(scale, d),
                                                  int(bool(causal)), _stream(stream)))


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, max_seqlen: int, causal: bool, scale=None, stream=None) -> None:
    T, H, d = q.shape
    nseq = cu_seqlens.numel() - 1
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _bf16(n, t, (T, H, d))
    _f32("lse", lse, (nseq, H, max_seqlen))
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
        raise ValueError("cu_seqlens must be a CUDA int32 tensor")
    _check("fa_fwd_varlen", lib().fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens),
                                                nseq, max_seqlen, T, H, d, _scale(scale, d), int(bool(causal)),
                                                _stream(stream)))


def fa_bwd_varlen_workspace_bytes(total: int, nseq: int, max_seqlen: int, H: int, d: int) -> int:
    return int(lib().fa_bwd_varlen_workspace_bytes(total, nseq, max_seqlen, H, d))


def fa_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_seqlens, max_seqlen: int, causal: bool,
                  scale=None, stream=None) -> None:
    T, H, d = q.shape
    nseq = cu_seqlens.numel() - 1
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv)):
        _bf16(n, t, (T, H, d))
    _f32("lse", lse, (nseq, H, max_seqlen))
    _check("fa_bwd_varlen", lib().fa_bwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(cu_seqlens), nseq, max_seqlen, T, H, d,
        _scale(scale, d), int(bool(causal)), _stream(stream)))


def _grouped(q, k, v, cu_seqlens):
    """Checks of q, k, v and cu_seqlens: (device, T, H, Hk, d, nseq, row strides)."""
    dev = _device_of("q", q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [T, H, d] and [T, Hk, d]")
    T, H, d = q.shape
    Hk = k.shape[1]
    ldq, ldk, ldv = _rows("q", q, T, H, d, dev), _rows("k", k, T, Hk, d, dev), _rows("v", v, T, Hk, d, dev)
    nseq = cu_seqlens.numel() - 1
    _dense("cu_seqlens", cu_seqlens, torch.int32, (nseq + 1,), dev)
    return dev, T, H, Hk, d, nseq, ldq, ldk, ldv


def _count(name: str, n: int) -> int:
    if not 0 <= n < 2 ** 31:
        raise ValueError(f"{name} must be an int32 count (got {n})")
    return n


def _launch_fwd_grouped(checked, q, k, v, o, lse, cu_seqlens, max_seqlen, causal, scale, stream, zero_tail) -> None:
    dev, T, H, Hk, d, nseq, ldq, ldk, ldv = checked
    _count("max_seqlen", max_seqlen)
    _check("fa_fwd_grouped", lib().fa_fwd_grouped(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), cu_seqlens.data_ptr(), nseq,
        max_seqlen, T, H, Hk, d, ldq, ldk, ldv, _scale(scale, d), bool(causal), zero_tail, _stream_of(stream, dev)))


def fa_fwd_grouped(q, k, v, o, lse, cu_seqlens, max_seqlen: int, causal: bool, scale=None, stream=None,
                   zero_tail: bool = False) -> None:
    """q, o [T, H, d], k, v [T, Hk, d] (rows of q, k, v may be slices of wider
    ones), lse fp32 [H, T]; query head h reads key/value head h // (H // Hk)."""
    checked = _grouped(q, k, v, cu_seqlens)
    dev, T, H, _, d = checked[:5]
    _dense("o", o, torch.bfloat16, (T, H, d), dev)
    _dense("lse", lse, torch.float32, (H, T), dev)
    _launch_fwd_grouped(checked, q, k, v, o, lse, cu_seqlens, max_seqlen, causal, scale, stream, bool(zero_tail))


def fa_bwd_grouped_workspace_bytes(nseq: int, max_seqlen: int, total: int, H: int, Hk: int, d: int,
                                   causal: bool) -> int:
    return lib().fa_bwd_grouped_workspace_bytes(nseq, max_seqlen, total, H, Hk, d, bool(causal))


def _launch_bwd_grouped(checked, q, k, v, o, dout, lse, dq, dk, dv, workspace, nbytes, cu_seqlens, max_seqlen, causal,
                        scale, stream, zero_tail) -> None:
    dev, T, H, Hk, d, nseq, ldq, ldk, ldv = checked
    _count("max_seqlen", max_seqlen)
    _dense("o", o, torch.bfloat16, (T, H, d), dev)
    _dense("dout", dout, torch.bfloat16, (T, H, d), dev)
    _dense("lse", lse, torch.float32, (H, T), dev)
    _check("fa_bwd_grouped", lib().fa_bwd_grouped(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(), dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), nbytes, cu_seqlens.data_ptr(), nseq, max_seqlen, T, H, Hk, d,
        ldq, ldk, ldv, _scale(scale, d), bool(causal), zero_tail, _stream_of(stream, dev)))


def fa_bwd_grouped(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_seqlens, max_seqlen: int, causal: bool,
                   scale=None, stream=None, zero_tail: bool = False) -> None:
    checked = _grouped(q, k, v, cu_seqlens)
    dev, T, H, Hk, d = checked[:5]
    _dense("dq", dq, torch.bfloat16, (T, H, d), dev)
    _dense("dk", dk, torch.bfloat16, (T, Hk, d), dev)
    _dense("dv", dv, torch.bfloat16, (T, Hk, d), dev)
    _launch_bwd_grouped(checked, q, k, v, o, dout, lse, dq, dk, dv, workspace, _nbytes(workspace, dev), cu_seqlens,
                        max_seqlen, causal, scale, stream, bool(zero_tail))


def _cache8(cache, dev: int):
    """Checks of a cache's four tensors: its page shape (num_blocks, Hk, block, d)."""
    k, v, k_scale, v_scale = cache
    shape = k.shape
    if len(shape) != 4:
        raise ValueError("cache pages must be [num_blocks, Hk, block, d]")
    _dense("cache.k", k, torch.float8_e4m3fn, shape, dev)
    _dense("cache.v", v, torch.float8_e4m3fn, shape, dev)
    _dense("cache.k_scale", k_scale, torch.float32, shape[:2], dev)
    _dense("cache.v_scale", v_scale, torch.float32, shape[:2], dev)
    return shape


def _block_table(t: torch.Tensor, rows: int, dev: int) -> int:
    if t.dim() != 2:
        raise ValueError("block_table must be [B, cols]")
    cols = t.shape[1]
    _dense("block_table", t, torch.int32, (rows, cols), dev)
    return cols


def fa_cache8_store(k, v, cache, block_table, cu_seqlens, start, max_new: int, stream=None) -> None:
    """Appends k, v [T, Hk, d] (rows may be slices of wider ones) to the cache
    (k, v, k_scale, v_scale): rows cu_seqlens[b] .. of sequence b become its
    tokens start[b], start[b] + 1, ..."""
    dev = _device_of("k", k)
    if k.dim() != 3:
        raise ValueError("k must be [T, Hk, d]")
    T, Hk, d = k.shape
    ldk, ldv = _rows("k", k, T, Hk, d, dev), _rows("v", v, T, Hk, d, dev)
    num_blocks, heads, block, dim = _cache8(cache, dev)
    if heads != Hk or dim != d:
        raise ValueError(f"the cache holds {heads} heads of {dim}, k and v have {Hk} of {d}")
    B = start.numel()
    cols = _block_table(block_table, B, dev)
    _dense("cu_seqlens", cu_seqlens, torch.int32, (B + 1,), dev)
    _dense("start", start, torch.int32, (B,), dev)
    _count("max_new", max_new)
    ck, cv, sk, sv = cache
    _check("fa_cache8_store", lib().fa_cache8_store(
        k.data_ptr(), v.data_ptr(), ck.data_ptr(), cv.data_ptr(), sk.data_ptr(), sv.data_ptr(), block_table.data_ptr(),
        cu_seqlens.data_ptr(), start.data_ptr(), B, max_new, T, num_blocks, cols, Hk, block, d, ldk, ldv,
        _stream_of(stream, dev)))


def fa_decode_cache8_workspace_bytes(B: int, Nq: int, H: int, Hk: int, max_seqlen: int, d: int) -> int:
    return lib().fa_decode_cache8_workspace_bytes(B, Nq, H, Hk, max_seqlen, d)


def _decode_cache8(q, cache, block_table, seqlens):
    """Checks of the inputs: (device, B, Nq, H, d, num_blocks, Hk, block, table columns)."""
    dev = _device_of("q", q)
    if q.dim() != 4:
        raise ValueError("q must be [B, Nq, H, d]")
    B, Nq, H, d = q.shape
    _dense("q", q, torch.bfloat16, q.shape, dev)
    num_blocks, Hk, block, dim = _cache8(cache, dev)
    if dim != d:
        raise ValueError(f"the cache holds heads of {dim}, q has {d}")
    cols = _block_table(block_table, B, dev)
    _dense("seqlens", seqlens, torch.int32, (B,), dev)
    return dev, B, Nq, H, d, num_blocks, Hk, block, cols


def _launch_decode_cache8(checked, q, cache, block_table, seqlens, o, lse, workspace, nbytes, max_seqlen, causal, scale,
                          stream) -> None:
    dev, B, Nq, H, d, num_blocks, Hk, block, cols = checked
    _count("max_seqlen", max_seqlen)
    ck, cv, sk, sv = cache
    _check("fa_fwd_decode_cache8", lib().fa_fwd_decode_cache8(
        q.data_ptr(), ck.data_ptr(), cv.data_ptr(), sk.data_ptr(), sv.data_ptr(), block_table.data_ptr(),
        seqlens.data_ptr(), o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), nbytes, B, Nq, H, Hk, num_blocks, cols,
        block, max_seqlen, d, _scale(scale, d), bool(causal), _stream_of(stream, dev)))


def fa_fwd_decode_cache8(q, cache, block_table, seqlens, o, lse, workspace, max_seqlen: int, causal: bool, scale=None,
                         stream=None) -> None:
    """q, o [B, Nq, H, d] over the cache (k, v, k_scale, v_scale); lse fp32 [B, H, Nq]."""
    checked = _decode_cache8(q, cache, block_table, seqlens)
    dev, B, Nq, H = checked[:4]
    _dense("o", o, torch.bfloat16, q.shape, dev)
    _dense("lse", lse, torch.float32, (B, H, Nq), dev)
    _launch_decode_cache8(checked, q, cache, block_table, seqlens, o, lse, workspace, _nbytes(workspace, dev), max_seqlen,
                          causal, scale, stream)


def _rotary(rotary, total: int, d: int, positions, dev: int):
    """Checks of a Rotary and its positions ([total] or [axes, total]; None where
    the call allows it): (pairs, axes, interleaved)."""
    turns, axis, axes, interleaved = rotary
    if turns.dim() != 1:
        raise ValueError("rotary.turns must be [pairs]")
    pairs = turns.numel()
    _dense("rotary.turns", turns, torch.int64, (pairs,), dev)
    _dense("rotary.axis", axis, torch.int32, (pairs,), dev)
    if pairs == 0 or pairs % 8 or 2 * pairs > d:
        raise ValueError(f"rotary: {pairs} pairs must be a multiple of 8 and at most half of a head's {d} dimensions")
    if not 1 <= axes <= pairs:
        raise ValueError(f"rotary: {axes} axes for {pairs} pairs")
    if positions is not None:
        _dense("positions", positions, torch.int32,
               (total,) if axes == 1 and positions.dim() == 1 else (axes, total), dev)
    return pairs, axes, bool(interleaved)


def _turn(q, k, positions, rotary):
    """Checks of fa_rotary's inputs: (device, T, H, Hk, d, pairs, axes, interleaved, row strides)."""
    dev = _device_of("q", q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [T, H, d] and [T, Hk, d]")
    T, H, d = q.shape
    Hk = k.shape[1]
    ldq, ldk = _rows("q", q, T, H, d, dev), _rows("k", k, T, Hk, d, dev)
    if positions is None:
        raise TypeError("positions must be an int32 tensor")
    return (dev, T, H, Hk, d, *_rotary(rotary, T, d, positions, dev), ldq, ldk)


def _launch_rotary(checked, q, k, q_out, k_out, positions, rotary, inverse, stream) -> None:
    dev, T, H, Hk, d, pairs, axes, interleaved, ldq, ldk = checked
    _check("fa_rotary", lib().fa_rotary(
        q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), positions.data_ptr(), rotary[0].data_ptr(),
        rotary[1].data_ptr(), T, H, Hk, d, pairs, axes, interleaved, inverse, ldq, ldk, _stream_of(stream, dev)))


def fa_rotary(q, k, q_out, k_out, positions, rotary, inverse: bool = False, stream=None) -> None:
    """q, q_out [T, H, d], k, k_out [T, Hk, d] (rows of q and k may be slices of
    wider ones); positions int32 [T] or [axes, T]."""
    checked = _turn(q, k, positions, rotary)
    dev, T, H, Hk, d = checked[:5]
    _dense("q_out", q_out, torch.bfloat16, (T, H, d), dev)
    _dense("k_out", k_out, torch.bfloat16, (T, Hk, d), dev)
    _launch_rotary(checked, q, k, q_out, k_out, positions, rotary, bool(inverse), stream)


def fa_cache8_store_rotary(q, k, v, q_out, cache, block_table, cu_seqlens, start, max_new: int, rotary, positions=None,
                           stream=None, zero_tail: bool = False) -> None:
    """fa_cache8_store of turned keys; q [T, H, d] turned into q_out."""
    dev = _device_of("q", q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [T, H, d] and [T, Hk, d]")
    T, H, d = q.shape
    Hk = k.shape[1]
    ldq, ldk, ldv = _rows("q", q, T, H, d, dev), _rows("k", k, T, Hk, d, dev), _rows("v", v, T, Hk, d, dev)
    _dense("q_out", q_out, torch.bfloat16, (T, H, d), dev)
    num_blocks, heads, block, dim = _cache8(cache, dev)
    if heads != Hk or dim != d:
        raise ValueError(f"the cache holds {heads} heads of {dim}, k and v have {Hk} of {d}")
    pairs, axes, interleaved = _rotary(rotary, T, d, positions, dev)
    B = start.numel()
    cols = _block_table(block_table, B, dev)
    _dense("cu_seqlens", cu_seqlens, torch.int32, (B + 1,), dev)
    _dense("start", start, torch.int32, (B,), dev)
    _count("max_new", max_new)
    ck, cv, sk, sv = cache
    _check("fa_cache8_store_rotary", lib().fa_cache8_store_rotary(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), ck.data_ptr(), cv.data_ptr(), sk.data_ptr(),
        sv.data_ptr(), block_table.data_ptr(), cu_seqlens.data_ptr(), start.data_ptr(),
        None if positions is None else positions.data_ptr(), rotary[0].data_ptr(), rotary[1].data_ptr(), B, max_new, T,
        num_blocks, cols, H, Hk, block, d, pairs, axes, interleaved, ldq, ldk, ldv, bool(zero_tail),
        _stream_of(stream, dev)))


def fa_chunk_cache8_workspace_bytes(B: int, max_new: int, total: int, H: int, Hk: int, max_seqlen: int, d: int) -> int:
    return lib().fa_chunk_cache8_workspace_bytes(B, max_new, total, H, Hk, max_seqlen, d)


def _chunk_cache8(q, cache, block_table, cu_seqlens, seqlens):
    """Checks of the inputs: (device, T, H, d, row stride, num_blocks, Hk, block, B, table columns)."""
    dev = _device_of("q", q)
    if q.dim() != 3:
        raise ValueError("q must be [T, H, d]")
    T, H, d = q.shape
    ldq = _rows("q", q, T, H, d, dev)
    num_blocks, Hk, block, dim = _cache8(cache, dev)
    if dim != d:
        raise ValueError(f"the cache holds heads of {dim}, q has {d}")
    B = seqlens.numel()
    cols = _block_table(block_table, B, dev)
    _dense("cu_seqlens", cu_seqlens, torch.int32, (B + 1,), dev)
    _dense("seqlens", seqlens, torch.int32, (B,), dev)
    return dev, T, H, d, ldq, num_blocks, Hk, block, B, cols


def _launch_chunk_cache8(checked, q, cache, block_table, cu_seqlens, seqlens, o, lse, workspace, nbytes, max_new,
                         max_seqlen, causal, scale, stream, zero_tail) -> None:
    dev, T, H, d, ldq, num_blocks, Hk, block, B, cols = checked
    _count("max_new", max_new)
    _count("max_seqlen", max_seqlen)
    ck, cv, sk, sv = cache
    _check("fa_fwd_chunk_cache8", lib().fa_fwd_chunk_cache8(
        q.data_ptr(), ck.data_ptr(), cv.data_ptr(), sk.data_ptr(), sv.data_ptr(), block_table.data_ptr(),
        cu_seqlens.data_ptr(), seqlens.data_ptr(), o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), nbytes, B, max_new,
        T, H, Hk, num_blocks, cols, block, max_seqlen, d, ldq, _scale(scale, d), bool(causal), zero_tail,
        _stream_of(stream, dev)))


def fa_fwd_chunk_cache8(q, cache, block_table, cu_seqlens, seqlens, o, lse, workspace, max_new: int, max_seqlen: int,
                        causal: bool, scale=None, stream=None, zero_tail: bool = False) -> None:
    """q, o [T, H, d] (rows of q may be slices of wider ones) over the cache (k, v,
    k_scale, v_scale); lse fp32 [H, T]."""
    checked = _chunk_cache8(q, cache, block_table, cu_seqlens, seqlens)
    dev, T, H, d = checked[:4]
    _dense("o", o, torch.bfloat16, (T, H, d), dev)
    _dense("lse", lse, torch.float32, (H, T), dev)
    _launch_chunk_cache8(checked, q, cache, block_table, cu_seqlens, seqlens, o, lse, workspace, _nbytes(workspace, dev),
                         max_new, max_seqlen, causal, scale, stream, bool(zero_tail))


def fa_decode_workspace_bytes(B: int, H: int, Nq: int, Nk: int, d: int) -> int:
    return int(lib().fa_decode_workspace_bytes(B, H, Nq, Nk, d))


def fa_fwd_decode(q, k, v, o, lse, workspace, causal: bool, scale=None, stream=None) -> None:
    B, Nq, H, d = q.shape
    Nk = k.shape[1]
    _bf16("q", q, (B, Nq, H, d))
    _bf16("o", o, (B, Nq, H, d))
    for n, t in (("k", k), ("v", v)):
        _bf16(n, t, (B, Nk, H, d))
    _f32("lse", lse, (B, H, Nq))
    _check("fa_fwd_decode", lib().fa_fwd_decode(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), B, H, Nq, Nk, d, _scale(scale, d), int(bool(causal)),
        _stream(stream)))


def fa_get_device_error(stream=None) -> int:
    return int(lib().fa_get_device_error(_stream(stream)))


def fa_cta_order(npairs: int, ntiles: int, slots: int):
    """Launch order of the attention kernels' CTAs (host only): returns
    (group, pair, tile) with pair[b], tile[b] the work item of launch index b."""
    import numpy as np

    group = ctypes.c_int(0)
    _check("fa_cta_order", lib().fa_cta_order(npairs, ntiles, slots, ctypes.byref(group), None, None, 0))
    n = -(-npairs // group.value) * group.value * ntiles
    pair, tile = np.zeros(n, dtype=np.int32), np.zeros(n, dtype=np.int32)
    _check("fa_cta_order", lib().fa_cta_order(npairs, ntiles, slots, None, pair.ctypes.data_as(_P),
                                              tile.ctypes.data_as(_P), n))
    return group.value, pair, tile


def fa_set_kernel_events(start_event, end_event) -> None:
    """Time the main kernel of the next backward call on this thread with two
    torch.cuda.Event objects (created with enable_timing=True)."""
    for ev in (start_event, end_event):
        # torch creates the underlying cudaEvent_t lazily, on the first
        # record; record once so there is a handle (and torch regards the
        # event as recorded).  The library records it again around the kernel.
        if ev is not None and ev.cuda_event == 0:
            ev.record()
    s = None if start_event is None else ctypes.c_void_p(start_event.cuda_event)
    e = None if end_event is None else ctypes.c_void_p(end_event.cuda_event)
    _check("fa_set_kernel_events", lib().fa_set_kernel_events(s, e))


def fa_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    return int(lib().fa_selftest_wait_timeout(int(limit_ns), _stream(stream)))


def fa_microbench(name: str, iters: int, stream=None) -> float:
    """Rate per SM per clock of one unit (see MICROBENCH for the names)."""
    out = ctypes.c_double(0.0)
    _check("fa_microbench", lib().fa_microbench(MICROBENCH[name], int(iters), ctypes.byref(out), _stream(stream)))
    return out.value
