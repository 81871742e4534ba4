"""ctypes binding of libpagedattn.so (argument marshalling only).

The functions named ``pa_*`` mirror the C entry points of ``include/pagedattn.h``
one to one: tensors are passed as their device pointers, sizes as ints, the
stream as the current torch CUDA stream unless one is given.  ``decode`` and
``write_cache`` derive the sizes from tensor shapes and call the same entry
points.  Every computation happens in the CUDA library; if it is missing the
first call raises, there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import torch

from .build import LIB_PATH

PA_OK = 0
PA_ERR_INVALID_ARG = -1
PA_ERR_UNSUPPORTED = -2
PA_ERR_CUDA = -3
PA_ERR_WORKSPACE = -4
PA_F32 = 0
PA_BF16 = 1
PA_FP8_E4M3 = 2
PA_DEVERR_BLOCK_ID = 1
PA_DEVERR_CONTEXT_LEN = 2
PA_DEVERR_SLOT = 4
PA_DEVERR_TIMEOUT = 8
PA_DEVERR_NO_BLOCKS = 16
PA_DEVERR_STATE = 32
PA_TABLES_RELEASE = -1

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
HEADER = os.path.join(INCLUDE, "pagedattn.h")
PA_ERR_NO_BLOCKS = -5


class PagedAttnError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"[{code}] {message}")
        self.code = code


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_SIGS = {
    "pa_decode": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _I]),
    "pa_decode_ws": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _I, _P, _SZ]),
    "pa_decode_ex": (
        _I,
        [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _I, _I, _P, _SZ, _I, _P],
    ),
    "pa_decode_append": (
        _I,
        [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _I, _I, _P, _SZ, _I, _P],
    ),
    "pa_decode_fp8_append": (
        _I,
        [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, ctypes.c_float, ctypes.c_float,
         _P, _I, _P, _SZ, _I, _P],
    ),
    "pa_decode_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "pa_decode_mq": (
        _I,
        [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _I, _I, _P, _SZ, _I, _P],
    ),
    "pa_decode_mq_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "pa_decode_mq_append": (
        _I,
        [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _I, _I, _P, _SZ, _I,
         _P],
    ),
    "pa_write_cache_fp8": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, ctypes.c_float, _P, _I, _P]),
    "pa_decode_fp8": (
        _I,
        [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, ctypes.c_float, ctypes.c_float, _P, _I,
         _P, _SZ, _I, _P],
    ),
    "pa_decode_fp8_mq": (
        _I,
        [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, ctypes.c_float, ctypes.c_float, _P,
         _I, _P, _SZ, _I, _P],
    ),
    "pa_decode_fp8_mq_append": (
        _I,
        [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, ctypes.c_float,
         ctypes.c_float, _P, _I, _P, _SZ, _I, _P],
    ),
    "pa_decode_static": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _I]),
    "pa_write_cache": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I]),
    "pa_write_cache_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _P]),
    "pa_last_error": (ctypes.c_char_p, []),
    "pa_bm_create": (_P, [_I, _I, _I, _I]),
    "pa_bm_destroy": (None, [_P]),
    "pa_bm_num_free_blocks": (_I, [_P]),
    "pa_bm_context_len": (_I, [_P, _I]),
    "pa_bm_ref_count": (_I, [_P, _I]),
    "pa_bm_append": (_I, [_P, _I, _I, _P, _P, _P]),
    "pa_bm_fork": (_I, [_P, _I, _I]),
    "pa_bm_append_batch": (_I, [_P, _I, _P, _P, _P, _P, _P, _P]),
    "pa_bm_share_prefix": (_I, [_P, _I, _I, _I]),
    "pa_bm_free": (_I, [_P, _I]),
    "pa_bm_export": (_I, [_P, _P, _P]),
    "pa_copy_blocks": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _I]),
    "pa_decode_mod": (
        _I,
        [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, ctypes.c_float, _P, _I, _P, _P, _P, _I,
         _I, _P, _SZ, _I, _P],
    ),
    "pa_decode_fp8_mod": (
        _I,
        [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, ctypes.c_float, ctypes.c_float,
         ctypes.c_float, _P, _I, _P, _P, _P, _I, _P, _SZ, _I, _P],
    ),
    "pa_decode_mod_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "pa_decode_prefix": (
        _I,
        [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _I, _I, _P, _SZ, _P],
    ),
    "pa_decode_fp8_prefix": (
        _I,
        [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, ctypes.c_float, ctypes.c_float,
         _P, _I, _P, _SZ, _P],
    ),
    "pa_decode_prefix_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "pa_tables_step": (_I, [_P] * 10 + [_I] * 6 + [_P, _P]),
    "pa_version": (_I, []),
    "pa_test_stall_copy": (_I, [ctypes.c_longlong, ctypes.c_uint]),
}


def library_path() -> str:
    return LIB_PATH


def load() -> ctypes.CDLL:
    """Load the shared library (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build the CUDA library first")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def header_symbols() -> list:
    """Names of the functions the public headers (include/*.h) declare."""
    names = set()
    for fn in sorted(os.listdir(INCLUDE)):
        if not fn.endswith(".h"):
            continue
        with open(os.path.join(INCLUDE, fn)) as f:
            text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
        names |= set(re.findall(r"\b(pa_\w+)\s*\(", text))
    return sorted(names)


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, torch.Tensor):
        return x.data_ptr()
    raise TypeError(f"expected a tensor or an int pointer, got {type(x)!r}")


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _made_for(stream, device, make):
    """``make()``, a tensor that a call on ``stream`` is to write: from that stream's memory, to which nothing still
    queued on the current stream writes, and in use on the current stream, whose work reads it, when it is freed."""
    if stream is None:
        return make()
    current = torch.cuda.current_stream(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))
    if stream.cuda_stream == current.cuda_stream:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(current)
    return t


def _check(rc: int) -> None:
    if rc != PA_OK:
        msg = load().pa_last_error()
        raise PagedAttnError(rc, msg.decode() if msg else "")


def dtype_code(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return PA_F32
    if dtype == torch.bfloat16:
        return PA_BF16
    raise ValueError(f"unsupported dtype {dtype}")


# ---- one-to-one entry points -------------------------------------------------
#
# The functions without the prefix pa_ take the pools' size from their shape and always
# give it to the library, so that tensor maps end with the pools and a block id
# outside them is skipped and reported (error_flag), never followed;
# check_block_ids=True says no more than that.


def pa_decode(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_heads, num_kv_heads,
              head_size, block_size, max_blocks_per_seq, scale, stream=None, dtype=None):
    dtype = dtype_code(query.dtype) if dtype is None else dtype
    _check(load().pa_decode(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                            _ptr(context_lens), num_seqs, num_heads, num_kv_heads, head_size, block_size,
                            max_blocks_per_seq, scale, _stream(stream), dtype))


def pa_decode_ws(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_heads, num_kv_heads,
                 head_size, block_size, max_blocks_per_seq, scale, stream, dtype, workspace, workspace_bytes):
    dtype = dtype_code(query.dtype) if dtype is None else dtype
    _check(load().pa_decode_ws(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                               _ptr(context_lens), num_seqs, num_heads, num_kv_heads, head_size, block_size,
                               max_blocks_per_seq, scale, _stream(stream), dtype, _ptr(workspace),
                               workspace_bytes))


def pa_decode_ex(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_heads, num_kv_heads,
                 head_size, block_size, max_blocks_per_seq, scale, stream=None, dtype=None,
                 num_physical_blocks=0, workspace=None, workspace_bytes=0, num_ranges=0, error_flag=None):
    dtype = dtype_code(query.dtype) if dtype is None else dtype
    _check(load().pa_decode_ex(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                               _ptr(context_lens), num_seqs, num_heads, num_kv_heads, head_size, block_size,
                               max_blocks_per_seq, scale, _stream(stream), dtype, num_physical_blocks,
                               _ptr(workspace), workspace_bytes, num_ranges, _ptr(error_flag)))


def pa_decode_static(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_heads, num_kv_heads,
                     head_size, block_size, max_blocks_per_seq, scale, stream=None, dtype=None):
    """pa_decode without any allocation: scratch is an array compiled into the library."""
    dtype = dtype_code(query.dtype) if dtype is None else dtype
    _check(load().pa_decode_static(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                   _ptr(context_lens), num_seqs, num_heads, num_kv_heads, head_size, block_size,
                                   max_blocks_per_seq, scale, _stream(stream), dtype))


def pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, num_ranges=0) -> int:
    return int(load().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, num_ranges))


def pa_decode_mq(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_queries, num_heads,
                 num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, stream=None, dtype=None,
                 num_physical_blocks=0, workspace=None, workspace_bytes=0, num_ranges=0, error_flag=None):
    dtype = dtype_code(query.dtype) if dtype is None else dtype
    _check(load().pa_decode_mq(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                               _ptr(context_lens), num_seqs, num_queries, num_heads, num_kv_heads, head_size,
                               block_size, max_blocks_per_seq, scale, _stream(stream), dtype, num_physical_blocks,
                               _ptr(workspace), workspace_bytes, num_ranges, _ptr(error_flag)))


def pa_decode_mq_workspace_size(num_seqs, num_queries, num_heads, num_kv_heads, head_size, num_ranges=0) -> int:
    return int(load().pa_decode_mq_workspace_size(num_seqs, num_queries, num_heads, num_kv_heads, head_size,
                                                  num_ranges))


def decode_multi(query, k_cache, v_cache, block_tables, context_lens, scale, out=None, stream=None, *,
                 num_ranges=0, workspace=None, error_flag=None, check_block_ids=False):
    """out[S, Q, H, D]: several causal query tokens per sequence (shapes as in ``pa_decode_mq``)."""
    _require_cuda(query, k_cache, v_cache, block_tables, context_lens, out, workspace, error_flag)
    S, Q, H, D = query.shape
    NB, bs, Hk, _ = k_cache.shape
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    pa_decode_mq(out, query, k_cache, v_cache, block_tables, context_lens, S, Q, H, Hk, D, bs,
                 block_tables.shape[1], float(scale), stream, dtype_code(query.dtype),
                 NB, workspace, ws_bytes, num_ranges, error_flag)
    return out


def pa_write_cache(k_new, v_new, slot_mapping, k_cache, v_cache, num_tokens, num_kv_heads, head_size,
                   block_size, num_physical_blocks, stream=None, dtype=None):
    dtype = dtype_code(k_new.dtype) if dtype is None else dtype
    _check(load().pa_write_cache(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
                                 num_tokens, num_kv_heads, head_size, block_size, num_physical_blocks,
                                 _stream(stream), dtype))


def pa_write_cache_ex(k_new, v_new, slot_mapping, k_cache, v_cache, num_tokens, num_kv_heads, head_size,
                      block_size, num_physical_blocks, stream=None, dtype=None, error_flag=None):
    dtype = dtype_code(k_new.dtype) if dtype is None else dtype
    _check(load().pa_write_cache_ex(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
                                    num_tokens, num_kv_heads, head_size, block_size, num_physical_blocks,
                                    _stream(stream), dtype, _ptr(error_flag)))


def pa_last_error() -> str:
    msg = load().pa_last_error()
    return msg.decode() if msg else ""


def pa_version() -> int:
    return int(load().pa_version())


def pa_test_stall_copy(tile: int, wait_limit_us: int = 0) -> None:
    """Test hook: the next decode launch on this thread withholds tile `tile`'s copies and bounds its waits."""
    _check(load().pa_test_stall_copy(tile, wait_limit_us))


# ---- shape-derived conveniences ---------------------------------------------


def _require_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def pa_decode_append(out, query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, num_seqs,
                     num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, stream=None,
                     dtype=None, num_physical_blocks=0, workspace=None, workspace_bytes=0, num_ranges=0,
                     error_flag=None):
    dtype = dtype_code(query.dtype) if dtype is None else dtype
    _check(load().pa_decode_append(_ptr(out), _ptr(query), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                   _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), num_seqs, num_heads,
                                   num_kv_heads, head_size, block_size, max_blocks_per_seq, float(scale),
                                   _stream(stream), dtype, num_physical_blocks, _ptr(workspace),
                                   workspace_bytes, num_ranges, _ptr(error_flag)))


def decode_append(query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale, out=None,
                  stream=None, *, num_ranges=0, workspace=None, error_flag=None, check_block_ids=False):
    """One decode step with the newest token's K/V (k_new/v_new[S, Hk, D]) written into the pools at
    position context_lens[s]-1 by the decode itself (shapes as in ``pa_decode_append``)."""
    _require_cuda(query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, out, workspace, error_flag)
    S, H, D = query.shape
    NB, bs, Hk, _ = k_cache.shape
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    pa_decode_append(out, query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, S, H, Hk, D, bs,
                     block_tables.shape[1], float(scale), stream, dtype_code(query.dtype),
                     NB, workspace, ws_bytes, num_ranges, error_flag)
    return out


def pa_decode_mq_append(out, query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, num_seqs,
                        num_queries, num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale,
                        stream=None, dtype=None, num_physical_blocks=0, workspace=None, workspace_bytes=0,
                        num_ranges=0, error_flag=None):
    dtype = dtype_code(query.dtype) if dtype is None else dtype
    _check(load().pa_decode_mq_append(_ptr(out), _ptr(query), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                      _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), num_seqs, num_queries,
                                      num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq,
                                      float(scale), _stream(stream), dtype, num_physical_blocks, _ptr(workspace),
                                      workspace_bytes, num_ranges, _ptr(error_flag)))


def decode_multi_append(query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale, out=None,
                        stream=None, *, num_ranges=0, workspace=None, error_flag=None, check_block_ids=False):
    """Several causal query tokens per sequence with their K/V (k_new/v_new[S*Q, Hk, D], token i of
    sequence s at row s*Q+i, position context_lens[s]-Q+i) written into the pools by the same launch
    (shapes as in ``pa_decode_mq_append``)."""
    _require_cuda(query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, out, workspace, error_flag)
    S, Q, H, D = query.shape
    NB, bs, Hk, _ = k_cache.shape
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    pa_decode_mq_append(out, query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, S, Q, H, Hk, D,
                        bs, block_tables.shape[1], float(scale), stream, dtype_code(query.dtype),
                        NB, workspace, ws_bytes, num_ranges, error_flag)
    return out


def decode_fp8_append(query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale, k_scale,
                      v_scale, out=None, stream=None, *, num_ranges=0, workspace=None, error_flag=None,
                      check_block_ids=False):
    """pa_decode_fp8_append: the FP8-pool step with the newest token's quantising write fused in."""
    _require_cuda(query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, out, workspace, error_flag)
    S, H, D = query.shape
    NB, bs, Hk, _ = k_cache.shape
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().pa_decode_fp8_append(_ptr(out), _ptr(query), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                       _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), S, H, Hk, D, bs,
                                       block_tables.shape[1], float(scale), float(k_scale), float(v_scale),
                                       _stream(stream), NB, _ptr(workspace), ws_bytes,
                                       num_ranges, _ptr(error_flag)))
    return out


def decode(query, k_cache, v_cache, block_tables, context_lens, scale, out=None, stream=None, *,
           num_ranges=0, workspace=None, error_flag=None, check_block_ids=False):
    """out[S, H, D] = paged decode attention (shapes as in ``pa_decode``)."""
    _require_cuda(query, k_cache, v_cache, block_tables, context_lens, out, workspace, error_flag)
    S, H, D = query.shape
    NB, bs, Hk, _ = k_cache.shape
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    pa_decode_ex(out, query, k_cache, v_cache, block_tables, context_lens, S, H, Hk, D, bs,
                 block_tables.shape[1], float(scale), stream, dtype_code(query.dtype),
                 NB, workspace, ws_bytes, num_ranges, error_flag)
    return out


def write_cache(k_new, v_new, slot_mapping, k_cache, v_cache, stream=None, *, error_flag=None):
    """Scatter k_new/v_new[T, Hk, D] into the pools at slot_mapping[T] (int64)."""
    _require_cuda(k_new, v_new, slot_mapping, k_cache, v_cache, error_flag)
    T, Hk, D = k_new.shape
    NB, bs = k_cache.shape[:2]
    pa_write_cache_ex(k_new, v_new, slot_mapping, k_cache, v_cache, T, Hk, D, bs, NB, stream,
                      dtype_code(k_new.dtype), error_flag)


def pa_copy_blocks(k_cache, v_cache, pairs, num_pairs, num_kv_heads, head_size, block_size, num_physical_blocks,
                   stream=None, dtype=None):
    dtype = dtype_code(k_cache.dtype) if dtype is None else dtype
    _check(load().pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(pairs), num_pairs, num_kv_heads, head_size,
                                 block_size, num_physical_blocks, _stream(stream), dtype))


class BlockManager:
    """The C block manager (pa_bm_*): host memory only, no device calls."""

    def __init__(self, num_blocks, block_size, max_seqs, max_blocks_per_seq):
        lib = load()
        self._h = lib.pa_bm_create(num_blocks, block_size, max_seqs, max_blocks_per_seq)
        if not self._h:
            raise PagedAttnError(PA_ERR_INVALID_ARG, pa_last_error())
        self.num_blocks, self.block_size = num_blocks, block_size
        self.max_seqs, self.max_blocks_per_seq = max_seqs, max_blocks_per_seq

    def close(self):
        if self._h:
            load().pa_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def num_free_blocks(self):
        return load().pa_bm_num_free_blocks(self._h)

    def context_len(self, seq):
        return load().pa_bm_context_len(self._h, seq)

    def ref_count(self, block):
        return load().pa_bm_ref_count(self._h, block)

    def append(self, seq, num_tokens):
        """Slots (int64 tensor) for num_tokens new tokens, and the list of (src, dst) block copies."""
        slots = torch.empty(max(num_tokens, 1), dtype=torch.int64)
        copies = (ctypes.c_int32 * 2)()
        n = ctypes.c_int(0)
        _check(load().pa_bm_append(self._h, seq, num_tokens, slots.data_ptr(), ctypes.addressof(copies),
                                   ctypes.addressof(n)))
        return slots[:num_tokens], [(copies[0], copies[1])] if n.value else []

    def append_batch(self, seqs, counts, slots_out=None, copies_out=None):
        """One call for many sequences; returns (slots, list of (src, dst) copies)."""
        seqs = torch.as_tensor(seqs, dtype=torch.int32)
        counts = torch.as_tensor(counts, dtype=torch.int32)
        total = int(counts.sum())
        if slots_out is None:
            slots_out = torch.empty(max(total, 1), dtype=torch.int64)
        if copies_out is None:
            copies_out = torch.empty(2 * max(len(seqs), 1), dtype=torch.int32)
        nc, nd = ctypes.c_int(0), ctypes.c_int(0)
        _check(load().pa_bm_append_batch(self._h, len(seqs), seqs.data_ptr(), counts.data_ptr(), slots_out.data_ptr(),
                                         copies_out.data_ptr(), ctypes.addressof(nc), ctypes.addressof(nd)))
        pairs = copies_out[: 2 * nc.value].view(-1, 2)
        return slots_out[:total], [tuple(p) for p in pairs.tolist()]

    def fork(self, parent, child):
        _check(load().pa_bm_fork(self._h, parent, child))

    def share_prefix(self, seq, donor, num_tokens):
        _check(load().pa_bm_share_prefix(self._h, seq, donor, num_tokens))

    def free(self, seq):
        _check(load().pa_bm_free(self._h, seq))

    def export(self):
        tables = torch.empty((self.max_seqs, self.max_blocks_per_seq), dtype=torch.int32)
        lens = torch.empty(self.max_seqs, dtype=torch.int32)
        _check(load().pa_bm_export(self._h, tables.data_ptr(), lens.data_ptr()))
        return tables, lens


def write_cache_fp8(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale, stream=None, *,
                    error_flag=None):
    """Quantise and scatter k_new/v_new[T, Hk, D] (bf16 or f32) into uint8 E4M3 pools."""
    _require_cuda(k_new, v_new, slot_mapping, k_cache, v_cache, error_flag)
    T, Hk, D = k_new.shape
    NB, bs = k_cache.shape[:2]
    _check(load().pa_write_cache_fp8(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), T,
                                     Hk, D, bs, NB, float(k_scale), float(v_scale), _stream(stream),
                                     dtype_code(k_new.dtype), _ptr(error_flag)))


def decode_fp8(query, k_cache, v_cache, block_tables, context_lens, scale, k_scale, v_scale, out=None, stream=None,
               *, num_ranges=0, workspace=None, error_flag=None, check_block_ids=False):
    """out[S, H, D] (bf16) over uint8 E4M3 pools."""
    _require_cuda(query, k_cache, v_cache, block_tables, context_lens, out, workspace, error_flag)
    S, H, D = query.shape
    NB, bs, Hk, _ = k_cache.shape
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().pa_decode_fp8(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                _ptr(context_lens), S, H, Hk, D, bs, block_tables.shape[1], float(scale),
                                float(k_scale), float(v_scale), _stream(stream), NB,
                                _ptr(workspace), ws_bytes, num_ranges, _ptr(error_flag)))
    return out


def decode_fp8_multi(query, k_cache, v_cache, block_tables, context_lens, scale, k_scale, v_scale, out=None,
                     stream=None, *, num_ranges=0, workspace=None, error_flag=None, check_block_ids=False):
    """out[S, Q, H, D] (bf16): several causal query tokens per sequence over uint8 E4M3 pools."""
    _require_cuda(query, k_cache, v_cache, block_tables, context_lens, out, workspace, error_flag)
    S, Q, H, D = query.shape
    NB, bs, Hk, _ = k_cache.shape
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().pa_decode_fp8_mq(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                   _ptr(context_lens), S, Q, H, Hk, D, bs, block_tables.shape[1], float(scale),
                                   float(k_scale), float(v_scale), _stream(stream), NB,
                                   _ptr(workspace), ws_bytes, num_ranges, _ptr(error_flag)))
    return out


def decode_fp8_multi_append(query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale, k_scale,
                            v_scale, out=None, stream=None, *, num_ranges=0, workspace=None, error_flag=None,
                            check_block_ids=False):
    """pa_decode_fp8_mq_append: the FP8 multi-query step with the Q new rows' quantising write fused in."""
    _require_cuda(query, k_new, v_new, k_cache, v_cache, block_tables, context_lens, out, workspace, error_flag)
    S, Q, H, D = query.shape
    NB, bs, Hk, _ = k_cache.shape
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().pa_decode_fp8_mq_append(_ptr(out), _ptr(query), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                          _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), S, Q, H, Hk, D, bs,
                                          block_tables.shape[1], float(scale), float(k_scale), float(v_scale),
                                          _stream(stream), NB, _ptr(workspace), ws_bytes,
                                          num_ranges, _ptr(error_flag)))
    return out


# ---- operators beyond plain decode ---------------------------------------------
#
# A step's small operators take a few microseconds on the GPU, so these
# functions check their tensors with few attribute reads and pass them on directly.


def _on(index, dtype, what, *ts):
    """Contiguous tensors of one type on CUDA device ``index`` (None: an argument left out)."""
    for t in ts:
        if t is not None and (t.dtype is not dtype or t.get_device() != index or not t.is_contiguous()):
            if t.dtype is not dtype:
                raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
            raise ValueError("tensors must be contiguous CUDA tensors on one device")


def _device_of(t):
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must be contiguous CUDA tensors on one device")
    return index


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, index):
    """cudaStream_t of ``stream`` (None: device ``index``'s current stream)."""
    if stream is None:
        return _raw_stream(index) if _raw_stream else torch.cuda.current_stream(index).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        if stream.device.index != index:
            raise ValueError("the stream belongs to another device than the tensors")
        return stream.cuda_stream
    return int(stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call_on(index, fn, *args):
    """One library call with the tensors' device current."""
    if _current_device() == index:
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc != PA_OK:
        _check(rc)


def pa_tables_step(block_tables, context_lens_out, seq_starts, slot_mapping, free_blocks, free_count_out,
                   context_lens, new_lens, free_count, prefix_table, num_prefix_blocks, num_seqs,
                   max_blocks_per_seq, block_size, num_physical_blocks, max_tokens, stream=None, error_flag=None):
    _check(load().pa_tables_step(_ptr(block_tables), _ptr(context_lens_out), _ptr(seq_starts), _ptr(slot_mapping),
                                 _ptr(free_blocks), _ptr(free_count_out), _ptr(context_lens), _ptr(new_lens),
                                 _ptr(free_count), _ptr(prefix_table), num_prefix_blocks, num_seqs,
                                 max_blocks_per_seq, block_size, num_physical_blocks, max_tokens, _stream(stream),
                                 _ptr(error_flag)))


def tables_step(block_tables, context_lens, new_lens, free_blocks, free_count, block_size, slot_mapping, *,
                prefix_table=None, context_lens_out=None, free_count_out=None, seq_starts=None, stream=None,
                error_flag=None):
    """One step's block tables and slots from the requests' lengths (as in ``pa_tables_step``).

    ``block_tables[S, MB]``, ``free_blocks[NB]`` and ``slot_mapping[T]`` (int64) are written in place; returns
    ``(context_lens_out[S], free_count_out[1], seq_starts[S + 1])``, which are not the inputs' buffers."""
    index = _device_of(block_tables)
    _on(index, torch.int32, "tables, lengths and the free list", block_tables, context_lens, new_lens, free_blocks,
        free_count, prefix_table, context_lens_out, free_count_out, seq_starts, error_flag)
    _on(index, torch.int64, "slot_mapping", slot_mapping)
    S, MB = block_tables.shape
    if context_lens.numel() != S or new_lens.numel() != S or free_count.numel() != 1:
        raise ValueError("context_lens and new_lens must have one entry per table row, free_count one entry")
    if context_lens_out is None:
        context_lens_out = _made_for(stream, context_lens.device, lambda: context_lens.new_empty(S))
    if free_count_out is None:
        free_count_out = _made_for(stream, context_lens.device, lambda: context_lens.new_empty(1))
    if seq_starts is None:
        seq_starts = _made_for(stream, context_lens.device, lambda: context_lens.new_empty(S + 1))
    if context_lens_out.numel() != S or free_count_out.numel() != 1 or seq_starts.numel() != S + 1:
        raise ValueError("context_lens_out, free_count_out and seq_starts must have S, 1 and S + 1 entries")
    _call_on(index, load().pa_tables_step, block_tables.data_ptr(), context_lens_out.data_ptr(),
             seq_starts.data_ptr(), slot_mapping.data_ptr(), free_blocks.data_ptr(), free_count_out.data_ptr(),
             context_lens.data_ptr(), new_lens.data_ptr(), free_count.data_ptr(),
             None if prefix_table is None else prefix_table.data_ptr(),
             0 if prefix_table is None else prefix_table.numel(), S, MB, block_size, free_blocks.numel(),
             slot_mapping.numel(), _stream_on(stream, index),
             None if error_flag is None else error_flag.data_ptr())
    return context_lens_out, free_count_out, seq_starts


def pa_decode_mod(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_queries, num_heads,
                  num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, softcap=0.0, alibi_slopes=None,
                  window=0, first_tokens=None, prefix_lens=None, stream=None, dtype=None, num_physical_blocks=0,
                  workspace=None, workspace_bytes=0, num_ranges=0, error_flag=None):
    dtype = dtype_code(query.dtype) if dtype is None else dtype
    _check(load().pa_decode_mod(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                _ptr(context_lens), num_seqs, num_queries, num_heads, num_kv_heads, head_size,
                                block_size, max_blocks_per_seq, scale, softcap, _ptr(alibi_slopes), window,
                                _ptr(first_tokens), _ptr(prefix_lens), _stream(stream), dtype, num_physical_blocks,
                                _ptr(workspace), workspace_bytes, num_ranges, _ptr(error_flag)))


def pa_decode_fp8_mod(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_queries, num_heads,
                      num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, k_scale, v_scale, softcap=0.0,
                      alibi_slopes=None, window=0, first_tokens=None, prefix_lens=None, stream=None,
                      num_physical_blocks=0, workspace=None, workspace_bytes=0, num_ranges=0, error_flag=None):
    _check(load().pa_decode_fp8_mod(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                    _ptr(context_lens), num_seqs, num_queries, num_heads, num_kv_heads, head_size,
                                    block_size, max_blocks_per_seq, scale, k_scale, v_scale, softcap,
                                    _ptr(alibi_slopes), window, _ptr(first_tokens), _ptr(prefix_lens),
                                    _stream(stream), num_physical_blocks, _ptr(workspace), workspace_bytes,
                                    num_ranges, _ptr(error_flag)))


def pa_decode_mod_workspace_size(num_seqs, num_queries, num_heads, num_kv_heads, head_size, kv_dtype,
                                 num_ranges=0) -> int:
    return int(load().pa_decode_mod_workspace_size(num_seqs, num_queries, num_heads, num_kv_heads, head_size,
                                                   kv_dtype, num_ranges))


def _step(query, k_cache, v_cache, block_tables, context_lens, out, pool_dtype):
    """(device index, S, Q, H, D, NB, bs, Hk, MB) of a step over paged pools, query [S, H, D] or [S, Q, H, D]."""
    index = query.get_device()
    if index < 0 or k_cache.get_device() != index or v_cache.get_device() != index or \
            block_tables.get_device() != index or context_lens.get_device() != index or not (
                query.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
                and block_tables.is_contiguous() and context_lens.is_contiguous()):
        raise ValueError("tensors must be contiguous CUDA tensors on one device")
    if k_cache.dtype is not pool_dtype or v_cache.dtype is not pool_dtype:
        raise ValueError(f"k_cache and v_cache must be {pool_dtype}, got {k_cache.dtype} and {v_cache.dtype}")
    if block_tables.dtype is not torch.int32 or context_lens.dtype is not torch.int32:
        raise ValueError("block_tables and context_lens must be torch.int32")
    shape = query.shape
    if len(shape) == 3:
        (S, H, D), Q = shape, 1
    else:
        S, Q, H, D = shape
    pool = k_cache.shape
    NB, bs, Hk, Dk = pool
    SB, MB = block_tables.shape
    if Dk != D or v_cache.shape != pool or SB != S or context_lens.numel() != S:
        raise ValueError("shapes of query, pools, block_tables and context_lens do not go together")
    if out is not None:
        _on(index, query.dtype, "out", out)
        if out.shape != shape:
            raise ValueError("out must have query's shape")
    return index, S, Q, H, D, NB, bs, Hk, MB


def _mod_pointers(index, S, H, alibi_slopes, first_tokens, prefix_lens):
    """Addresses of the optional per-head and per-sequence arrays."""
    slopes = first = prefix = None
    if alibi_slopes is not None:
        _on(index, torch.float32, "alibi_slopes", alibi_slopes)
        if alibi_slopes.numel() != H:
            raise ValueError("alibi_slopes must have one entry per query head")
        slopes = alibi_slopes.data_ptr()
    if first_tokens is not None:
        _on(index, torch.int32, "first_tokens", first_tokens)
        if first_tokens.numel() != S:
            raise ValueError("first_tokens must have one entry per sequence")
        first = first_tokens.data_ptr()
    if prefix_lens is not None:
        _on(index, torch.int32, "prefix_lens", prefix_lens)
        if prefix_lens.numel() != S:
            raise ValueError("prefix_lens must have one entry per sequence")
        prefix = prefix_lens.data_ptr()
    return slopes, first, prefix


def _scratch_pointers(index, workspace, error_flag):
    """(address and bytes of the workspace, address of the error word)."""
    ws, ws_bytes, err = None, 0, None
    if workspace is not None:
        _on(index, workspace.dtype, "workspace", workspace)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if error_flag is not None:
        _on(index, torch.int32, "error_flag", error_flag)
        err = error_flag.data_ptr()
    return ws, ws_bytes, err


def decode_mod(query, k_cache, v_cache, block_tables, context_lens, scale, out=None, stream=None, *, softcap=0.0,
               alibi_slopes=None, window=0, first_tokens=None, prefix_lens=None, num_ranges=0, workspace=None,
               error_flag=None, check_block_ids=False):
    """Decode with capped, biased and masked scores (as in ``pa_decode_mod``); query and out [S, H, D] or [S, Q, H, D]."""
    dtype = query.dtype
    index, S, Q, H, D, NB, bs, Hk, MB = _step(query, k_cache, v_cache, block_tables, context_lens, out, dtype)
    code = dtype_code(dtype)
    slopes, first, prefix = _mod_pointers(index, S, H, alibi_slopes, first_tokens, prefix_lens)
    ws, ws_bytes, err = _scratch_pointers(index, workspace, error_flag)
    raw = _stream_on(stream, index)
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    _call_on(index, load().pa_decode_mod, out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
             block_tables.data_ptr(), context_lens.data_ptr(), S, Q, H, Hk, D, bs, MB, scale, softcap, slopes, window,
             first, prefix, raw, code, NB, ws, ws_bytes, num_ranges, err)
    return out


def decode_fp8_mod(query, k_cache, v_cache, block_tables, context_lens, scale, k_scale, v_scale, out=None,
                   stream=None, *, softcap=0.0, alibi_slopes=None, window=0, first_tokens=None, prefix_lens=None,
                   num_ranges=0, workspace=None, error_flag=None, check_block_ids=False):
    """``decode_mod`` over uint8 E4M3 pools (as in ``pa_decode_fp8_mod``)."""
    if query.dtype is not torch.bfloat16:
        raise ValueError(f"query must be {torch.bfloat16}, got {query.dtype}")
    index, S, Q, H, D, NB, bs, Hk, MB = _step(query, k_cache, v_cache, block_tables, context_lens, out, torch.uint8)
    slopes, first, prefix = _mod_pointers(index, S, H, alibi_slopes, first_tokens, prefix_lens)
    ws, ws_bytes, err = _scratch_pointers(index, workspace, error_flag)
    raw = _stream_on(stream, index)
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    _call_on(index, load().pa_decode_fp8_mod, out.data_ptr(), query.data_ptr(), k_cache.data_ptr(),
             v_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), S, Q, H, Hk, D, bs, MB, scale,
             k_scale, v_scale, softcap, slopes, window, first, prefix, raw, NB, ws, ws_bytes,
             num_ranges, err)
    return out


def pa_decode_prefix(out, query, k_cache, v_cache, prefix_table, block_tables, context_lens, num_seqs, num_queries,
                     num_heads, num_kv_heads, head_size, block_size, num_prefix_blocks, max_blocks_per_seq, scale,
                     stream=None, dtype=None, num_physical_blocks=0, workspace=None, workspace_bytes=0,
                     error_flag=None):
    dtype = dtype_code(query.dtype) if dtype is None else dtype
    _check(load().pa_decode_prefix(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(prefix_table),
                                   _ptr(block_tables), _ptr(context_lens), num_seqs, num_queries, num_heads,
                                   num_kv_heads, head_size, block_size, num_prefix_blocks, max_blocks_per_seq, scale,
                                   _stream(stream), dtype, num_physical_blocks, _ptr(workspace), workspace_bytes,
                                   _ptr(error_flag)))


def pa_decode_fp8_prefix(out, query, k_cache, v_cache, prefix_table, block_tables, context_lens, num_seqs, num_queries,
                         num_heads, num_kv_heads, head_size, block_size, num_prefix_blocks, max_blocks_per_seq, scale,
                         k_scale, v_scale, stream=None, num_physical_blocks=0, workspace=None, workspace_bytes=0,
                         error_flag=None):
    _check(load().pa_decode_fp8_prefix(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache), _ptr(prefix_table),
                                       _ptr(block_tables), _ptr(context_lens), num_seqs, num_queries, num_heads,
                                       num_kv_heads, head_size, block_size, num_prefix_blocks, max_blocks_per_seq,
                                       scale, k_scale, v_scale, _stream(stream), num_physical_blocks, _ptr(workspace),
                                       workspace_bytes, _ptr(error_flag)))


def pa_decode_prefix_workspace_size(num_seqs, num_queries, num_heads, num_kv_heads, head_size) -> int:
    return int(load().pa_decode_prefix_workspace_size(num_seqs, num_queries, num_heads, num_kv_heads, head_size))


def decode_prefix(query, k_cache, v_cache, prefix_table, block_tables, context_lens, scale, out=None, stream=None, *,
                  workspace=None, error_flag=None, check_block_ids=False):
    """Decode of a batch that shares the prefix in the blocks ``prefix_table[NP]``, attended once for all (as in
    ``pa_decode_prefix``); query and out [S, H, D] or [S, Q, H, D]."""
    dtype = query.dtype
    index, S, Q, H, D, NB, bs, Hk, MB = _step(query, k_cache, v_cache, block_tables, context_lens, out, dtype)
    code = dtype_code(dtype)
    _on(index, torch.int32, "prefix_table", prefix_table)
    ws, ws_bytes, err = _scratch_pointers(index, workspace, error_flag)
    raw = _stream_on(stream, index)
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    _call_on(index, load().pa_decode_prefix, out.data_ptr(), query.data_ptr(), k_cache.data_ptr(),
             v_cache.data_ptr(), prefix_table.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), S, Q, H,
             Hk, D, bs, prefix_table.numel(), MB, scale, raw, code, NB, ws, ws_bytes, err)
    return out


def decode_fp8_prefix(query, k_cache, v_cache, prefix_table, block_tables, context_lens, scale, k_scale, v_scale,
                      out=None, stream=None, *, workspace=None, error_flag=None, check_block_ids=False):
    """``decode_prefix`` over uint8 E4M3 pools (as in ``pa_decode_fp8_prefix``)."""
    if query.dtype is not torch.bfloat16:
        raise ValueError(f"query must be {torch.bfloat16}, got {query.dtype}")
    index, S, Q, H, D, NB, bs, Hk, MB = _step(query, k_cache, v_cache, block_tables, context_lens, out, torch.uint8)
    _on(index, torch.int32, "prefix_table", prefix_table)
    ws, ws_bytes, err = _scratch_pointers(index, workspace, error_flag)
    raw = _stream_on(stream, index)
    if out is None:
        out = _made_for(stream, query.device, lambda: torch.empty_like(query))
    _call_on(index, load().pa_decode_fp8_prefix, out.data_ptr(), query.data_ptr(), k_cache.data_ptr(),
             v_cache.data_ptr(), prefix_table.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), S, Q, H,
             Hk, D, bs, prefix_table.numel(), MB, scale, k_scale, v_scale, raw, NB, ws,
             ws_bytes, err)
    return out
