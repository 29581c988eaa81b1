"""Paged MLA decode attention for one GB300 (sm_103a): the Python binding of
libmla_gb300, whose C ABI is declared in include/mla.h.

The binding only marshals arguments: it checks tensor dtypes, shapes and
devices, passes raw pointers and the current CUDA stream to the library, and
turns status codes into exceptions.  Every step of the computation runs in
the library's CUDA kernels.  There is no fallback: if the library cannot be
loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import build as _build

__all__ = [
    "MLAError", "Dims", "dims", "load_library", "check_dims", "cache_append", "auto_num_splits",
    "decode_workspace_size", "decode", "decode_multi_workspace_size", "decode_multi", "decode_sparse_workspace_size",
    "decode_sparse", "cache_read", "expand_kv", "prompt_attention_workspace_size", "prompt_attention",
    "decode_no_alloc", "combine", "read_device_status", "read_status_word",
    "set_timing_events", "status_string", "version",
    "MLA_OK", "MLA_ERR_INVALID_ARG", "MLA_ERR_UNSUPPORTED", "MLA_ERR_WORKSPACE", "MLA_ERR_CUDA",
    "MLA_ERR_DEVICE_TIMEOUT", "MLA_ERR_DEVICE_BOUNDS", "MLA_CACHE_BF16", "MLA_CACHE_INT8", "MLA_CACHE_FP8",
    "MLA_CACHE_FP4", "FP4_ROW_BYTES", "MAX_Q_LEN", "MAX_TOP_K", "MAX_PREFILL_CHUNK", "MAX_PROMPT_SEQS",
]

MLA_OK = 0
MLA_ERR_INVALID_ARG = -1
MLA_ERR_UNSUPPORTED = -2
MLA_ERR_WORKSPACE = -3
MLA_ERR_CUDA = -4
MLA_ERR_DEVICE_TIMEOUT = -5
MLA_ERR_DEVICE_BOUNDS = -6
MLA_CACHE_BF16 = 0
MLA_CACHE_INT8 = 1
MLA_CACHE_FP8 = 2
MLA_CACHE_FP4 = 4
FP4_ROW_BYTES = 320  # MLA_FP4_ROW_BYTES in include/mla.h
MAX_Q_LEN = 8  # MLA_MAX_Q_LEN in include/mla.h
MAX_PREFILL_CHUNK = 2048  # MLA_MAX_PREFILL_CHUNK in include/mla.h
MAX_TOP_K = 1 << 20  # MLA_MAX_TOP_K in include/mla.h
MAX_PROMPT_SEQS = 1 << 20  # MLA_MAX_PROMPT_SEQS in include/mla.h

# every function include/mla.h declares
EXPORTED_SYMBOLS = (
    "mla_check_dims", "mla_cache_append", "mla_auto_num_splits", "mla_decode_workspace_size",
    "mla_decode", "mla_combine", "mla_read_device_status", "mla_read_status_word",
    "mla_status_string", "mla_set_timing_events", "mla_version", "mla_decode_no_alloc",
    "mla_test_inject_wait_timeout", "mla_decode_multi_workspace_size", "mla_decode_multi",
    "mla_decode_sparse_workspace_size", "mla_decode_sparse", "mla_test_force_single_cta",
    "mla_prefill_workspace_size", "mla_prefill", "mla_cache_read", "mla_expand_kv",
    "mla_prompt_attention_workspace_size", "mla_prompt_attention",
)
NO_ALLOC_WORKSPACE_BYTES = 16 << 20  # MLA_NO_ALLOC_WORKSPACE_BYTES in include/mla.h


class MLAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("kv_lora_rank", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("qk_nope_dim", ctypes.c_int32),
                ("v_head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("cache_dtype", ctypes.c_int32)]


def dims(num_heads: int, page_size: int, int8: bool = False, kv_lora_rank: int = 512, rope_dim: int = 64,
         qk_nope_dim: int = 128, v_head_dim: int = 128, fp8: bool = False, fp4: bool = False) -> Dims:
    """Model dimensions; ``int8`` / ``fp8`` select a 1-byte cache (INT8 codes, or
    FP8 E4M3 codes held as uint8 or torch.float8_e4m3fn) with per-token scales,
    ``fp4`` one of FP4 rows (uint8 [pages, page_size, FP4_ROW_BYTES]: E2M1 codes
    and their scales, no scale tensor)."""
    if bool(int8) + bool(fp8) + bool(fp4) > 1:
        raise ValueError("int8, fp8 and fp4 are exclusive")
    code = MLA_CACHE_INT8 if int8 else MLA_CACHE_FP8 if fp8 else MLA_CACHE_FP4 if fp4 else MLA_CACHE_BF16
    return Dims(num_heads, kv_lora_rank, rope_dim, qk_nope_dim, v_head_dim, page_size, code)


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int32


def load_library(build_if_missing: bool = False, path: str | None = None):
    """Load libmla_gb300.so (building it first if asked and it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB_PATH
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m mla_decode_attention_paged_gb300.build`")
    lib = ctypes.CDLL(path)
    DP = ctypes.POINTER(Dims)
    sig = {
        "mla_check_dims": (_I, [DP]),
        "mla_cache_append": (_I, [DP, _P, _P, _I, _P, _I, _I, _P, _P, _I, _P, _P, ctypes.c_double, _P, _P]),
        "mla_auto_num_splits": (_I, [DP, _I]),
        "mla_decode_workspace_size": (ctypes.c_size_t, [DP, _I, _I]),
        "mla_decode": (_I, [DP, _P, _P, _P, _P, _I, _P, _I, _P, _I, _P, _P, ctypes.c_float, _I, _P,
                            ctypes.c_size_t, _P, _P, _P]),
        "mla_decode_multi_workspace_size": (ctypes.c_size_t, [DP, _I, _I, _I]),
        "mla_decode_multi": (_I, [DP, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _P, _P, ctypes.c_float, _I, _P,
                                  ctypes.c_size_t, _P, _P, _P]),
        "mla_decode_sparse_workspace_size": (ctypes.c_size_t, [DP, _I, _I, _I]),
        "mla_decode_sparse": (_I, [DP, _P, _P, _P, _P, _I, _P, _I, _P, _I, _P, _I, _P, _P, ctypes.c_float, _I, _P,
                                   ctypes.c_size_t, _P, _P, _P]),
        "mla_decode_no_alloc": (_I, [DP, _P, _P, _P, _P, _I, _P, _I, _P, _I, _P, _P, ctypes.c_float, _I, _P, _P,
                                     _P, _P]),
        "mla_combine": (_I, [DP, _P, _P, _I, _I, _P, _P, _P]),
        "mla_read_device_status": (_I, [_P, ctypes.POINTER(ctypes.c_int32), _P]),
        "mla_read_status_word": (_I, [_P, ctypes.POINTER(ctypes.c_int32), _P]),
        "mla_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "mla_set_timing_events": (_I, [_P, _P]),
        "mla_version": (ctypes.c_int, []),
        "mla_test_inject_wait_timeout": (_I, [_I]),
        "mla_test_force_single_cta": (_I, [_I]),
        "mla_prefill_workspace_size": (ctypes.c_size_t, [DP, _I, _I, _I]),
        "mla_prefill": (_I, [DP, _P, _P, _I, _P, _I, _P, _I, _I, _P, _P, ctypes.c_double, _P, _P, _P, _P,
                             ctypes.c_float, _I, _P, ctypes.c_size_t, _P, _P, _P]),
        "mla_cache_read": (_I, [DP, _P, _P, _I, _P, _I, _I, _P, _P, _I, _P, _P, _P, _P]),
        "mla_expand_kv": (_I, [DP, _P, _I, _P, _P, _P, _P, _P, _P]),
        "mla_prompt_attention_workspace_size": (ctypes.c_size_t, [DP, _I, _I]),
        "mla_prompt_attention": (_I, [DP, _P, _P, _I, _P, _P, _P, _I, _I, _P, _P, _I, ctypes.c_float, _P,
                                      ctypes.c_size_t, _P, _P, _P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _L():
    return _lib if _lib is not None else load_library()


def status_string(status: int) -> str:
    return _L().mla_status_string(int(status)).decode()


def version() -> int:
    return _L().mla_version()


def _check(status: int, what: str):
    if status != MLA_OK:
        raise MLAError(status, what)


def _ptr(t: torch.Tensor | None, dtype=None, name="tensor", device=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on(t: torch.Tensor, dtype, index: int, name: str) -> int:
    """Pointer of a contiguous tensor of this type on CUDA device ``index`` (_ptr
    with its common case first: these checks are most of a small call's host time)."""
    try:
        if t.dtype is dtype and t.get_device() == index and index >= 0 and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    return _ptr(t, dtype, name, torch.device("cuda", index) if index >= 0 else None)


def _holds(t: torch.Tensor, dtype, index: int, name: str, n: int) -> int:
    """_on of a tensor with at least the ``n`` elements that the call reads or writes."""
    try:
        if t.dtype is dtype and t.numel() >= n and t.get_device() == index and index >= 0 and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    p = _on(t, dtype, index, name)  # raises what is wrong, unless it is the size
    if t.numel() < n:
        raise ValueError(f"{name} has {t.numel()} elements, the call needs {n}")
    return p


def _index(t: torch.Tensor, name: str = "q_nope") -> int:
    """CUDA device of a tensor."""
    if _ptr(t, None, name) is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    return t.get_device()


# num_heads, kv_lora_rank, rope_dim, qk_nope_dim, v_head_dim, page_size and cache_dtype of a
# Dims at once (cheaper than four fields by their names).
_fields = struct.Struct("=7i").unpack_from


def _workspace(t: torch.Tensor, index: int) -> tuple[int, int]:
    """Pointer and bytes of a workspace tensor of any type."""
    try:
        if t.get_device() == index and index >= 0 and t.is_contiguous():
            return t.data_ptr(), t.nbytes
    except AttributeError:
        pass
    return _on(t, t.dtype if isinstance(t, torch.Tensor) else None, index, "workspace"), t.nbytes


# The type of a cache tensor by mla_cache_dtype, where it is not bf16.
_CODES = {MLA_CACHE_INT8: torch.int8, MLA_CACHE_FP8: torch.uint8, MLA_CACHE_FP4: torch.uint8}


def _cache_ptrs(code: int, page: int, width: int, cache: torch.Tensor, scale_zero: torch.Tensor | None, index: int):
    """Pointers of the cache rows (bf16 values, int8 codes, E4M3 codes, or FP4
    rows) and of their per-token scales (None for bf16 and FP4 caches)."""
    if code == MLA_CACHE_FP4:
        p, s = _on(cache, torch.uint8, index, "cache"), cache.shape
        if len(s) != 3 or s[1] != page or s[2] != FP4_ROW_BYTES:
            raise ValueError(f"cache must have shape [pages, {page}, {FP4_ROW_BYTES}], got {list(s)}")
        return p, None
    if code == MLA_CACHE_FP8 and isinstance(cache, torch.Tensor) and cache.dtype == torch.float8_e4m3fn:
        cache = cache.view(torch.uint8)
    rows = cache.shape[0] * page
    p = _holds(cache, _CODES.get(code, torch.bfloat16), index, "cache", rows * width)
    if code == MLA_CACHE_BF16 or scale_zero is None:  # without its scales the library refuses a 1-byte cache
        return p, None
    return p, _holds(scale_zero, torch.float32, index, "scale_zero", rows * (2 if code == MLA_CACHE_INT8 else 1))


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def check_dims(d: Dims) -> int:
    return _L().mla_check_dims(ctypes.byref(d))


def cache_append(d: Dims, cache: torch.Tensor, scale_zero: torch.Tensor | None, block_table: torch.Tensor,
                 seq_ids: torch.Tensor, positions: torch.Tensor, c_kv: torch.Tensor, k_pe: torch.Tensor,
                 rope_theta: float = 10000.0, device_status: torch.Tensor | None = None, stream=None) -> None:
    """mla_cache_append: write new tokens' rows into the paged cache (in place)."""
    _, R, rope, _, _, P, code = _fields(d)
    dev, at, i32, bf16 = cache.device, cache.get_device(), torch.int32, torch.bfloat16
    cache_p, scale_p = _cache_ptrs(code, P, R + rope, cache, scale_zero, at)
    table_p, table = _on(block_table, i32, at, "block_table"), block_table.shape
    ids_p, n = _on(seq_ids, i32, at, "seq_ids"), seq_ids.numel()
    st = _call_on(
        dev, stream, _L().mla_cache_append, ctypes.byref(d), cache_p, scale_p, cache.shape[0], table_p,
        table[0], table[1], ids_p, _holds(positions, i32, at, "positions", n), n,
        _holds(c_kv, bf16, at, "c_kv", n * R), _holds(k_pe, bf16, at, "k_pe", n * rope), float(rope_theta),
        None if device_status is None else _on(device_status, i32, at, "device_status"))
    _check(st, "mla_cache_append")


def auto_num_splits(d: Dims, batch: int) -> int:
    n = _L().mla_auto_num_splits(ctypes.byref(d), int(batch))
    if n < 0:
        raise MLAError(n, "mla_auto_num_splits")
    return n


def decode_workspace_size(d: Dims, batch: int, num_splits: int = 0) -> int:
    n = _L().mla_decode_workspace_size(ctypes.byref(d), int(batch), int(num_splits))
    if n == 0:
        raise MLAError(MLA_ERR_INVALID_ARG, "mla_decode_workspace_size")
    return n


def decode(d: Dims, q_nope, q_pe, cache, scale_zero, block_table, seq_lens, W_UK, W_UV, softmax_scale: float,
           num_splits: int = 0, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
           lse_out: torch.Tensor | None = None, want_lse: bool = True, stream=None):
    """mla_decode: one decode step; returns (out bf16 [B, H, 128], lse fp32 [B, H] or None).

    If ``workspace`` is None a uint8 buffer of the required size is taken from
    torch's allocator here (the library itself never allocates)."""
    H, R, rope, nope, vdim, P, code = _fields(d)
    B = q_nope.shape[0]
    dev = q_nope.device
    if workspace is None:
        workspace = _new(decode_workspace_size(d, B, num_splits), torch.uint8, dev, stream)
    if out is None:
        out = _new((B, H, vdim), torch.bfloat16, dev, stream)
    if lse_out is None and want_lse:
        lse_out = _new((B, H), torch.float32, dev, stream)
    at, i32, bf16 = q_nope.get_device(), torch.int32, torch.bfloat16
    rows, max_pages = B * H, block_table.shape[1]
    st = _call_on(
        dev, stream, _L().mla_decode, ctypes.byref(d), _holds(q_nope, bf16, at, "q_nope", rows * nope),
        _holds(q_pe, bf16, at, "q_pe", rows * rope), *_cache_ptrs(code, P, R + rope, cache, scale_zero, at),
        cache.shape[0], _holds(block_table, i32, at, "block_table", B * max_pages), max_pages,
        _holds(seq_lens, i32, at, "seq_lens", B), B,
        _holds(W_UK, bf16, at, "W_UK", H * nope * R), _holds(W_UV, bf16, at, "W_UV", H * vdim * R),
        float(softmax_scale), int(num_splits), *_workspace(workspace, at), _holds(out, bf16, at, "out", rows * vdim),
        None if lse_out is None else _holds(lse_out, torch.float32, at, "lse_out", rows))
    _check(st, "mla_decode")
    return out, lse_out


def decode_multi_workspace_size(d: Dims, batch: int, q_len: int, num_splits: int = 0) -> int:
    n = _L().mla_decode_multi_workspace_size(ctypes.byref(d), int(batch), int(q_len), int(num_splits))
    if n == 0:
        raise MLAError(MLA_ERR_INVALID_ARG, "mla_decode_multi_workspace_size")
    return n


def decode_multi(d: Dims, q_nope, q_pe, cache, scale_zero, block_table, seq_lens, W_UK, W_UV,
                 softmax_scale: float, num_splits: int = 0, workspace: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, lse_out: torch.Tensor | None = None, want_lse: bool = True,
                 stream=None):
    """mla_decode_multi: q_len = q_nope.shape[1] query tokens per sequence (the
    last q_len tokens of each cache, causal among themselves); q_nope bf16
    [B, T, H, 128], q_pe bf16 [B, T, H, 64].  Returns (out bf16 [B, T, H, 128],
    lse fp32 [B, T, H] or None)."""
    H, R, rope, nope, vdim, P, code = _fields(d)
    B, T = q_nope.shape[0], q_nope.shape[1]
    dev = q_nope.device
    if workspace is None:
        workspace = _new(decode_multi_workspace_size(d, B, T, num_splits), torch.uint8, dev, stream)
    if out is None:
        out = _new((B, T, H, vdim), torch.bfloat16, dev, stream)
    if lse_out is None and want_lse:
        lse_out = _new((B, T, H), torch.float32, dev, stream)
    at, i32, bf16 = q_nope.get_device(), torch.int32, torch.bfloat16
    rows, max_pages = B * T * H, block_table.shape[1]
    st = _call_on(
        dev, stream, _L().mla_decode_multi, ctypes.byref(d), _holds(q_nope, bf16, at, "q_nope", rows * nope),
        _holds(q_pe, bf16, at, "q_pe", rows * rope), *_cache_ptrs(code, P, R + rope, cache, scale_zero, at),
        cache.shape[0], _holds(block_table, i32, at, "block_table", B * max_pages), max_pages,
        _holds(seq_lens, i32, at, "seq_lens", B), B, T,
        _holds(W_UK, bf16, at, "W_UK", H * nope * R), _holds(W_UV, bf16, at, "W_UV", H * vdim * R),
        float(softmax_scale), int(num_splits), *_workspace(workspace, at), _holds(out, bf16, at, "out", rows * vdim),
        None if lse_out is None else _holds(lse_out, torch.float32, at, "lse_out", rows))
    _check(st, "mla_decode_multi")
    return out, lse_out


def prefill_workspace_size(d: Dims, batch: int, chunk: int, num_splits: int = 0) -> int:
    n = _L().mla_prefill_workspace_size(ctypes.byref(d), int(batch), int(chunk), int(num_splits))
    if n == 0:
        raise MLAError(MLA_ERR_INVALID_ARG, "mla_prefill_workspace_size")
    return n


def prefill(d: Dims, cache, scale_zero, block_table, seq_lens, c_kv, k_pe, q_nope, q_pe, W_UK, W_UV,
            softmax_scale: float, rope_theta: float = 10000.0, num_splits: int = 0,
            workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
            lse_out: torch.Tensor | None = None, want_lse: bool = True, stream=None):
    """mla_prefill: one chunk of chunk = q_nope.shape[1] tokens per sequence,
    at positions seq_lens[b] - chunk .. seq_lens[b] - 1.  Writes c_kv bf16
    [B, chunk, 512] / k_pe bf16 [B, chunk, 64] into the cache, then attends
    q_nope bf16 [B, chunk, H, 128] / q_pe [B, chunk, H, 64] causally.  Returns
    (out bf16 [B, chunk, H, 128], lse fp32 [B, chunk, H] or None)."""
    H, R, rope, nope, vdim, P, code = _fields(d)
    B, T = q_nope.shape[0], q_nope.shape[1]
    dev = q_nope.device
    if workspace is None:
        workspace = _new(prefill_workspace_size(d, B, T, num_splits), torch.uint8, dev, stream)
    if out is None:
        out = _new((B, T, H, vdim), torch.bfloat16, dev, stream)
    if lse_out is None and want_lse:
        lse_out = _new((B, T, H), torch.float32, dev, stream)
    at, i32, bf16 = q_nope.get_device(), torch.int32, torch.bfloat16
    cache_p, scale_p = _cache_ptrs(code, P, R + rope, cache, scale_zero, at)
    rows, max_pages = B * T * H, block_table.shape[1]
    st = _call_on(
        dev, stream, _L().mla_prefill, ctypes.byref(d), cache_p, scale_p, cache.shape[0],
        _holds(block_table, i32, at, "block_table", B * max_pages), max_pages,
        _holds(seq_lens, i32, at, "seq_lens", B), B, T,
        _holds(c_kv, bf16, at, "c_kv", B * T * R), _holds(k_pe, bf16, at, "k_pe", B * T * rope),
        float(rope_theta), _holds(q_nope, bf16, at, "q_nope", rows * nope),
        _holds(q_pe, bf16, at, "q_pe", rows * rope), _holds(W_UK, bf16, at, "W_UK", H * nope * R),
        _holds(W_UV, bf16, at, "W_UV", H * vdim * R), float(softmax_scale), int(num_splits), *_workspace(workspace, at),
        _holds(out, bf16, at, "out", rows * vdim),
        None if lse_out is None else _holds(lse_out, torch.float32, at, "lse_out", rows))
    _check(st, "mla_prefill")
    return out, lse_out


def decode_sparse_workspace_size(d: Dims, batch: int, top_k: int, num_splits: int = 0) -> int:
    n = _L().mla_decode_sparse_workspace_size(ctypes.byref(d), int(batch), int(top_k), int(num_splits))
    if n == 0:
        raise MLAError(MLA_ERR_INVALID_ARG, "mla_decode_sparse_workspace_size")
    return n


def decode_sparse(d: Dims, q_nope, q_pe, cache, scale_zero, block_table, seq_lens, token_indices, W_UK, W_UV,
                  softmax_scale: float, num_splits: int = 0, workspace: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, lse_out: torch.Tensor | None = None, want_lse: bool = True,
                  stream=None):
    """mla_decode_sparse: attention over the listed positions of each sequence
    (token_indices int32 [B, top_k], -1 = padding).  Returns (out bf16
    [B, H, 128], lse fp32 [B, H] or None)."""
    H, R, rope, nope, vdim, P, code = _fields(d)
    B, K = token_indices.shape
    dev = q_nope.device
    if workspace is None:
        workspace = _new(decode_sparse_workspace_size(d, B, K, num_splits), torch.uint8, dev, stream)
    if out is None:
        out = _new((B, H, vdim), torch.bfloat16, dev, stream)
    if lse_out is None and want_lse:
        lse_out = _new((B, H), torch.float32, dev, stream)
    at, i32, bf16 = q_nope.get_device(), torch.int32, torch.bfloat16
    rows, max_pages = B * H, block_table.shape[1]
    st = _call_on(
        dev, stream, _L().mla_decode_sparse, ctypes.byref(d), _holds(q_nope, bf16, at, "q_nope", rows * nope),
        _holds(q_pe, bf16, at, "q_pe", rows * rope), *_cache_ptrs(code, P, R + rope, cache, scale_zero, at),
        cache.shape[0], _holds(block_table, i32, at, "block_table", B * max_pages), max_pages,
        _holds(seq_lens, i32, at, "seq_lens", B), B, _on(token_indices, i32, at, "token_indices"), K,
        _holds(W_UK, bf16, at, "W_UK", H * nope * R), _holds(W_UV, bf16, at, "W_UV", H * vdim * R),
        float(softmax_scale), int(num_splits), *_workspace(workspace, at), _holds(out, bf16, at, "out", rows * vdim),
        None if lse_out is None else _holds(lse_out, torch.float32, at, "lse_out", rows))
    _check(st, "mla_decode_sparse")
    return out, lse_out


def _arg(t: torch.Tensor, name: str, dtype, shape: tuple, dev: torch.device) -> int:
    """Pointer of a contiguous tensor of this type, shape and device."""
    try:  # the common case first: these checks are most of a small call's host time
        if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    p = _ptr(t, dtype, name, dev)  # raises what is wrong, unless it is the shape
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    return p


def _dims_of(t: torch.Tensor, name: str, n: int):
    """Shape of an ``n``-dimensional CUDA tensor (the sizes the other arguments are checked against)."""
    try:
        s = t.shape
        if len(s) == n and t.is_cuda:
            return s
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {list(t.shape)}")
    raise ValueError(f"{name} must be a CUDA tensor")


def _call_on(dev: torch.device, stream, fn, *args) -> int:
    """fn(*args, stream) with ``dev`` current, on ``stream`` or dev's current stream."""
    if dev.index != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return fn(*args, _stream(stream))
    return fn(*args, torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else _stream(stream))


def _new(shape, dtype, dev: torch.device, stream) -> torch.Tensor:
    """torch.empty in the memory of the stream that the call runs on: a tensor
    of another stream's memory could still be in use there, or be handed out
    again there while the call runs."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):  # handle 0 is the default stream: ExternalStream(0) is another
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def cache_read(d: Dims, cache: torch.Tensor, scale_zero: torch.Tensor | None, block_table: torch.Tensor,
               cu_rows: torch.Tensor, starts: torch.Tensor | None = None, n_rows: int | None = None,
               c_kv: torch.Tensor | None = None, k_pe: torch.Tensor | None = None,
               device_status: torch.Tensor | None = None, stream=None):
    """mla_cache_read: the cached rows of a packed batch, dequantised to bf16.
    Sequence b's rows are cu_rows[b] .. cu_rows[b + 1] - 1 of the outputs, read
    from position starts[b] (0 without ``starts``) on.  Returns (c_kv bf16
    [n_rows, 512], k_pe bf16 [n_rows, 64]); ``n_rows`` may be left out where
    an output is given."""
    i32, bf16 = torch.int32, torch.bfloat16
    pages, page, row = _dims_of(cache, "cache", 3)
    B, max_pages = _dims_of(block_table, "block_table", 2)
    dev, P = cache.device, d.page_size
    at = dev.index
    if n_rows is None:
        given = c_kv if c_kv is not None else k_pe
        if given is None:
            raise ValueError("n_rows is needed where neither c_kv nor k_pe is given")
        n_rows = _dims_of(given, "c_kv" if c_kv is not None else "k_pe", 2)[0]
    if c_kv is None:
        c_kv = _new((n_rows, d.kv_lora_rank), bf16, dev, stream)
    if k_pe is None:
        k_pe = _new((n_rows, d.rope_dim), bf16, dev, stream)
    code = d.cache_dtype
    if code == MLA_CACHE_FP8 and cache.dtype == torch.float8_e4m3fn:
        cache = cache.view(torch.uint8)
    want = _CODES.get(code, bf16)
    width = FP4_ROW_BYTES if code == MLA_CACHE_FP4 else d.kv_lora_rank + d.rope_dim
    st = _call_on(
        dev, stream, _L().mla_cache_read, ctypes.byref(d),
        _on(cache, want, at, "cache") if page == P and row == width else _arg(cache, "cache", want, (pages, P, width), dev),
        None if code in (MLA_CACHE_BF16, MLA_CACHE_FP4) else
        _arg(scale_zero, "scale_zero", torch.float32, (pages, P, 2) if code == MLA_CACHE_INT8 else (pages, P), dev),
        pages, _on(block_table, i32, at, "block_table"), B, max_pages,
        None if starts is None else _arg(starts, "starts", i32, (B,), dev),
        _arg(cu_rows, "cu_rows", i32, (B + 1,), dev), int(n_rows),
        _arg(c_kv, "c_kv", bf16, (n_rows, d.kv_lora_rank), dev),
        _arg(k_pe, "k_pe", bf16, (n_rows, d.rope_dim), dev),
        None if device_status is None else _ptr(device_status, torch.int32, "device_status", dev))
    _check(st, "mla_cache_read")
    return c_kv, k_pe


def expand_kv(d: Dims, c_kv: torch.Tensor, W_UK: torch.Tensor, W_UV: torch.Tensor, k_nope: torch.Tensor | None = None,
              v: torch.Tensor | None = None, device_status: torch.Tensor | None = None, stream=None):
    """mla_expand_kv: latents c_kv bf16 [n, 512] to per-head keys and values.
    Returns (k_nope bf16 [n, H, 128], v bf16 [n, H, 128])."""
    n = _dims_of(c_kv, "c_kv", 2)[0]
    dev, H, R, bf16 = c_kv.device, d.num_heads, d.kv_lora_rank, torch.bfloat16
    if k_nope is None:
        k_nope = _new((n, H, d.qk_nope_dim), bf16, dev, stream)
    if v is None:
        v = _new((n, H, d.v_head_dim), bf16, dev, stream)
    st = _call_on(dev, stream, _L().mla_expand_kv, ctypes.byref(d), _arg(c_kv, "c_kv", bf16, (n, R), dev), n,
                  _arg(W_UK, "W_UK", bf16, (H, d.qk_nope_dim, R), dev),
                  _arg(W_UV, "W_UV", bf16, (H, d.v_head_dim, R), dev),
                  _arg(k_nope, "k_nope", bf16, (n, H, d.qk_nope_dim), dev),
                  _arg(v, "v", bf16, (n, H, d.v_head_dim), dev),
                  None if device_status is None else _ptr(device_status, torch.int32, "device_status", dev))
    _check(st, "mla_expand_kv")
    return k_nope, v


def prompt_attention_workspace_size(d: Dims, num_seqs: int, n_q: int) -> int:
    n = _L().mla_prompt_attention_workspace_size(ctypes.byref(d), int(num_seqs), int(n_q))
    if n == 0:
        raise MLAError(MLA_ERR_INVALID_ARG, "mla_prompt_attention_workspace_size")
    return n


def prompt_attention(d: Dims, q_nope: torch.Tensor, q_pe: torch.Tensor, k_nope: torch.Tensor, k_pe: torch.Tensor,
                     v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor, softmax_scale: float,
                     workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     lse_out: torch.Tensor | None = None, want_lse: bool = True, stream=None):
    """mla_prompt_attention: causal attention of packed queries q_nope bf16
    [n_q, H, 128], q_pe [n_q, H, 64] over packed keys k_nope bf16 [n_k, H_kv,
    128], k_pe [n_k, 64] and values v [n_k, H_kv, 128]; sequence b has the
    query rows cu_q[b] .. cu_q[b + 1] - 1 and the key rows cu_k[b] ..
    cu_k[b + 1] - 1, its queries being its last positions.  Returns (out bf16
    [n_q, H, 128], lse fp32 [n_q, H] or None)."""
    n_q = _dims_of(q_nope, "q_nope", 3)[0]
    n_k, kv_heads, _ = _dims_of(k_nope, "k_nope", 3)
    B = _dims_of(cu_q, "cu_q", 1)[0] - 1
    dev, H, bf16 = q_nope.device, d.num_heads, torch.bfloat16
    if workspace is None:
        workspace = _new(prompt_attention_workspace_size(d, B, n_q), torch.uint8, dev, stream)
    if out is None:
        out = _new((n_q, H, d.v_head_dim), bf16, dev, stream)
    if lse_out is None and want_lse:
        lse_out = _new((n_q, H), torch.float32, dev, stream)
    st = _call_on(
        dev, stream, _L().mla_prompt_attention, ctypes.byref(d),
        _arg(q_nope, "q_nope", bf16, (n_q, H, d.qk_nope_dim), dev),
        _arg(q_pe, "q_pe", bf16, (n_q, H, d.rope_dim), dev), n_q,
        _arg(k_nope, "k_nope", bf16, (n_k, kv_heads, d.qk_nope_dim), dev),
        _arg(k_pe, "k_pe", bf16, (n_k, d.rope_dim), dev), _arg(v, "v", bf16, (n_k, kv_heads, d.v_head_dim), dev), n_k,
        kv_heads, _arg(cu_q, "cu_q", torch.int32, (B + 1,), dev), _arg(cu_k, "cu_k", torch.int32, (B + 1,), dev), B,
        float(softmax_scale), _ptr(workspace, None, "workspace", dev), workspace.nbytes,
        _arg(out, "out", bf16, (n_q, H, d.v_head_dim), dev),
        None if lse_out is None else _arg(lse_out, "lse_out", torch.float32, (n_q, H), dev))
    _check(st, "mla_prompt_attention")
    return out, lse_out


def decode_no_alloc(d: Dims, q_nope, q_pe, cache, scale_zero, block_table, seq_lens, W_UK, W_UV,
                    softmax_scale: float, num_splits: int = 0, out: torch.Tensor | None = None,
                    lse_out: torch.Tensor | None = None, device_status: torch.Tensor | None = None, stream=None):
    """mla_decode_no_alloc: mla_decode on the library's fixed scratch array, for
    callers that cannot allocate device memory (outputs are still the
    caller's).  Returns (out, lse)."""
    H, R, rope, nope, vdim, P, code = _fields(d)
    B = q_nope.shape[0]
    dev = q_nope.device
    if out is None:
        out = _new((B, H, vdim), torch.bfloat16, dev, stream)
    at, i32, bf16 = q_nope.get_device(), torch.int32, torch.bfloat16
    rows, max_pages = B * H, block_table.shape[1]
    st = _call_on(
        dev, stream, _L().mla_decode_no_alloc, ctypes.byref(d), _holds(q_nope, bf16, at, "q_nope", rows * nope),
        _holds(q_pe, bf16, at, "q_pe", rows * rope), *_cache_ptrs(code, P, R + rope, cache, scale_zero, at),
        cache.shape[0], _holds(block_table, i32, at, "block_table", B * max_pages), max_pages,
        _holds(seq_lens, i32, at, "seq_lens", B), B,
        _holds(W_UK, bf16, at, "W_UK", H * nope * R), _holds(W_UV, bf16, at, "W_UV", H * vdim * R),
        float(softmax_scale), int(num_splits),
        _holds(out, bf16, at, "out", rows * vdim),
        None if lse_out is None else _holds(lse_out, torch.float32, at, "lse_out", rows),
        None if device_status is None else _on(device_status, i32, at, "device_status"))
    _check(st, "mla_decode_no_alloc")
    return out, lse_out


def combine(d: Dims, partial_o: torch.Tensor, partial_lse: torch.Tensor, o_lat_out=None, lse_out=None,
            stream=None):
    """mla_combine over [B, S, H, 512] partials; returns (o_lat [B, H, 512], lse [B, H])."""
    B, S, H, D = partial_o.shape
    dev = partial_o.device
    if o_lat_out is None:
        o_lat_out = _new((B, H, D), torch.float32, dev, stream)
    if lse_out is None:
        lse_out = _new((B, H), torch.float32, dev, stream)
    at, f32 = _index(partial_o, "partial_o"), torch.float32
    rows = B * d.num_heads
    st = _call_on(
        dev, stream, _L().mla_combine, ctypes.byref(d),
        _holds(partial_o, f32, at, "partial_o", rows * S * d.kv_lora_rank),
        _holds(partial_lse, f32, at, "partial_lse", rows * S), B, S,
        _holds(o_lat_out, f32, at, "o_lat_out", rows * d.kv_lora_rank), _holds(lse_out, f32, at, "lse_out", rows))
    _check(st, "mla_combine")
    return o_lat_out, lse_out


def read_device_status(workspace: torch.Tensor, stream=None) -> int:
    v, at = ctypes.c_int32(0), _index(workspace, "workspace")
    p, _ = _workspace(workspace, at)
    _check(_call_on(workspace.device, stream, _L().mla_read_device_status, p, ctypes.byref(v)), "mla_read_device_status")
    return v.value


def read_status_word(word: torch.Tensor, stream=None) -> int:
    v, p = ctypes.c_int32(0), _on(word, torch.int32, _index(word, "status word"), "status word")
    _check(_call_on(word.device, stream, _L().mla_read_status_word, p, ctypes.byref(v)), "mla_read_status_word")
    return v.value


def test_inject_wait_timeout(enable: bool) -> None:
    """Test hook: make the attention kernel's first page wait of each CTA unsatisfiable
    (it times out and the status word reports MLA_ERR_DEVICE_TIMEOUT)."""
    _check(_L().mla_test_inject_wait_timeout(1 if enable else 0), "mla_test_inject_wait_timeout")


def test_force_single_cta(enable: bool) -> None:
    """Test hook: run bf16 decodes on the single-CTA attention kernel (the
    fallback for devices that cannot place CTA pairs)."""
    _check(_L().mla_test_force_single_cta(1 if enable else 0), "mla_test_force_single_cta")


def set_timing_events(start: torch.cuda.Event | None, stop: torch.cuda.Event | None) -> None:
    """Have mla_decode record these events around its attention kernel (None clears)."""
    a = start.cuda_event if start is not None else None
    b = stop.cuda_event if stop is not None else None
    _check(_L().mla_set_timing_events(a, b), "mla_set_timing_events")
