"""ctypes binding of libpaged_gqa.so: argument marshalling only."""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional

import torch

from . import build as _build

PG_BF16, PG_F16, PG_E4M3, PG_I32, PG_F32, PG_FP4 = 1, 2, 3, 4, 5, 6
STATUS_NAMES = {0: "PG_OK", -1: "PG_ERR_INVALID_ARG", -2: "PG_ERR_UNSUPPORTED", -3: "PG_ERR_CUDA",
                -4: "PG_ERR_TIMEOUT", -5: "PG_ERR_DEVICE_BOUNDS", -6: "PG_ERR_WORKSPACE"}

# Every symbol include/paged_gqa.h declares.
EXPORTED = ("paged_gqa_attn", "paged_gqa_attn_ex", "paged_gqa_attn_noalloc", "paged_gqa_attn_quant_q",
            "paged_gqa_sparse_attn", "paged_gqa_cache_write",
            "paged_gqa_cache_write_fp4", "paged_gqa_cache_read_fp4", "paged_gqa_attn_fp4", "paged_gqa_attn_fp4_ex",
            "paged_gqa_rope",
            "paged_gqa_build_tables", "paged_gqa_tree_masks", "paged_gqa_attn_tree", "paged_gqa_attn_tree_ex",
            "paged_gqa_cache_keep", "paged_gqa_attn_prompt", "paged_gqa_attn_prompt_ex",
            "paged_gqa_prompt_workspace_size",
            "paged_gqa_workspace_size",
            "paged_gqa_last_error",
            "paged_gqa_check_device_errors", "paged_gqa_set_path", "paged_gqa_set_stall_test", "paged_gqa_last_plan",
            "paged_gqa_set_kernel_events", "paged_gqa_version")


class PagedGQAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class PgTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


_lock = threading.Lock()
_lib = None

# Descriptors are packed into a per-thread array of pg_tensor and passed by address: one
# struct.pack_into per tensor, by its number of dims, instead of a ctypes Structure built field
# by field.
_DESC_FMT = [struct.Struct(f"=Qii{n}q{8 * (4 - n)}x{n}q{8 * (4 - n)}x") for n in range(5)]
assert all(ctypes.sizeof(PgTensor) == f.size == 80 for f in _DESC_FMT)
_PACK_INTO = [f.pack_into for f in _DESC_FMT]
_tls = threading.local()


def _desc_buf():
    b = getattr(_tls, "buf", None)
    if b is None:
        arr = (PgTensor * 13)()
        base = ctypes.addressof(arr)
        b = _tls.buf = (arr, [base + 80 * i for i in range(13)], memoryview(arr).cast("B"))
    return b


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load the library (building it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if build_if_missing:
                _build.build()
            if not os.path.exists(_build.LIB):
                raise RuntimeError(f"libpaged_gqa.so not found at {_build.LIB}; run paged_gqa_gb300.build")
            lib = ctypes.CDLL(_build.LIB)
            P = ctypes.c_void_p  # descriptors are passed as addresses (see _pack)
            f, c_vp = ctypes.c_float, ctypes.c_void_p
            lib.paged_gqa_attn.argtypes = [P, P, P, P, P, P, f, f, f, P, c_vp]
            lib.paged_gqa_attn.restype = ctypes.c_int
            lib.paged_gqa_attn_ex.argtypes = [P, P, P, P, P, P, f, f, f, f, P, c_vp, ctypes.c_size_t, c_vp]
            lib.paged_gqa_attn_ex.restype = ctypes.c_int
            lib.paged_gqa_cache_write.argtypes = [P, P, P, P, P, P, P, f, f, c_vp]
            lib.paged_gqa_attn_quant_q.restype = ctypes.c_int
            lib.paged_gqa_attn_quant_q.argtypes = [P, P, P, P, P, P, f, f, f, P, c_vp]
            lib.paged_gqa_sparse_attn.restype = ctypes.c_int
            lib.paged_gqa_sparse_attn.argtypes = [P, P, P, P, P, P, P, f, f, f, P, c_vp]
            lib.paged_gqa_cache_write.restype = ctypes.c_int
            lib.paged_gqa_cache_write_fp4.argtypes = [P, P, P, P, P, P, P, f, f, c_vp]
            lib.paged_gqa_cache_read_fp4.argtypes = [P, P, P, P, P, f, f, P, P, c_vp]
            lib.paged_gqa_attn_fp4.argtypes = [P, P, P, P, P, P, f, f, f, P, c_vp]
            lib.paged_gqa_attn_fp4_ex.argtypes = [P, P, P, P, P, P, f, f, f, P, c_vp, ctypes.c_size_t, c_vp]
            lib.paged_gqa_rope.argtypes = [P, P, P, P, ctypes.POINTER(ctypes.c_int32), ctypes.c_int, ctypes.c_int, P, P, c_vp]
            lib.paged_gqa_build_tables.argtypes = [P, P, P, ctypes.c_int] + [P] * 10 + [c_vp]
            lib.paged_gqa_tree_masks.argtypes = [P, P, P, P, P, c_vp]
            lib.paged_gqa_attn_tree.argtypes = [P, P, P, P, P, P, P, f, f, f, P, c_vp]
            lib.paged_gqa_attn_tree_ex.argtypes = [P, P, P, P, P, P, P, f, f, f, P, c_vp, ctypes.c_size_t, c_vp]
            lib.paged_gqa_cache_keep.argtypes = [P, P, P, P, P, P, P, P, c_vp]
            lib.paged_gqa_attn_prompt.argtypes = [P, P, P, P, f, P, P, c_vp]
            lib.paged_gqa_attn_prompt_ex.argtypes = [P, P, P, P, f, P, P, c_vp, ctypes.c_size_t, c_vp]
            lib.paged_gqa_prompt_workspace_size.argtypes = [ctypes.c_int] * 5
            lib.paged_gqa_prompt_workspace_size.restype = ctypes.c_size_t
            for name in ("cache_write_fp4", "cache_read_fp4", "attn_fp4", "attn_fp4_ex", "rope", "build_tables", "tree_masks",
                         "attn_tree", "attn_tree_ex", "cache_keep", "attn_prompt", "attn_prompt_ex"):
                getattr(lib, "paged_gqa_" + name).restype = ctypes.c_int
            lib.paged_gqa_workspace_size.argtypes = [ctypes.c_int] * 7
            lib.paged_gqa_workspace_size.restype = ctypes.c_size_t
            lib.paged_gqa_last_error.restype = ctypes.c_char_p
            lib.paged_gqa_check_device_errors.argtypes = [c_vp]
            lib.paged_gqa_check_device_errors.restype = ctypes.c_int
            lib.paged_gqa_set_path.argtypes = [ctypes.c_int]
            lib.paged_gqa_set_path.restype = ctypes.c_int
            lib.paged_gqa_set_stall_test.argtypes = [ctypes.c_uint32]
            lib.paged_gqa_set_stall_test.restype = ctypes.c_int
            lib.paged_gqa_last_plan.argtypes = [ctypes.POINTER(ctypes.c_int64)]
            lib.paged_gqa_last_plan.restype = ctypes.c_int
            lib.paged_gqa_version.restype = ctypes.c_int
            lib.paged_gqa_set_kernel_events.argtypes = [ctypes.c_int, c_vp, c_vp]
            lib.paged_gqa_set_kernel_events.restype = ctypes.c_int
            _lib = lib
    return _lib


def exported_symbols():
    lib = load()
    return {name: hasattr(lib, name) for name in EXPORTED}


_DTYPES = {torch.bfloat16: PG_BF16, torch.float16: PG_F16, torch.int32: PG_I32, torch.float32: PG_F32,
           torch.uint8: PG_E4M3}
if hasattr(torch, "float8_e4m3fn"):
    _DTYPES[torch.float8_e4m3fn] = PG_E4M3
_DTYPES_FP4 = {**_DTYPES, torch.uint8: PG_FP4}  # in the 4-bit calls uint8 is a 4-bit cache


def _desc(t: Optional[torch.Tensor], dtype: Optional[int] = None) -> PgTensor:
    """pg_tensor view of a torch tensor (uint8 is read as e4m3 bit patterns)."""
    d = PgTensor()
    if t is None:
        return d
    if t.dim() > 4:
        raise ValueError("at most 4 dims")
    d.data = t.data_ptr() if t.numel() > 0 else 0
    d.dtype = dtype if dtype is not None else _DTYPES[t.dtype]
    d.ndim = t.dim()
    for i in range(t.dim()):
        d.shape[i] = t.shape[i]
        d.stride[i] = t.stride(i)
    return d


def _pack(*tensors, dtypes=_DTYPES):
    """Addresses of pg_tensor descriptors of the given tensors, valid until the next call
    from this thread (the library copies what it needs before it returns)."""
    _, addresses, mv = _desc_buf()
    off = 0
    for t in tensors:
        sh = t.shape
        n = len(sh)
        if n > 4:
            raise ValueError("at most 4 dims")
        # (the data pointer of a tensor without elements is 0)
        _PACK_INTO[n](mv, off, t.data_ptr(), dtypes[t.dtype], n, *sh, *t.stride())
        off += 80
    return addresses[:len(tensors)]


# The current stream's handle without a Stream object around it (2.5 us less per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int):
    if status != 0:
        msg = load().paged_gqa_last_error().decode(errors="replace")
        raise PagedGQAError(status, msg)


def paged_gqa_attn(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, k_descale: float,
                   v_descale: float, softmax_scale: float, out, stream=None) -> None:
    """out[T, Hq, 256] (bf16) = paged GQA attention; see include/paged_gqa.h."""
    lib = load()
    d = _pack(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, out)
    _check(lib.paged_gqa_attn(*d[:6], float(k_descale), float(v_descale), float(softmax_scale), d[6],
                              _stream(stream)))


def paged_gqa_attn_ex(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, q_descale: float,
                      k_descale: float, v_descale: float, softmax_scale: float, out, workspace,
                      stream=None) -> None:
    """Same as paged_gqa_attn with q_descale and a caller-owned workspace tensor."""
    lib = load()
    d = _pack(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, out)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    ptr = workspace.data_ptr() if workspace is not None else None
    _check(lib.paged_gqa_attn_ex(*d[:6], float(q_descale), float(k_descale), float(v_descale),
                                 float(softmax_scale), d[6], ptr, nbytes, _stream(stream)))


def paged_gqa_attn_quant_q(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, k_descale: float,
                           v_descale: float, softmax_scale: float, out, stream=None) -> None:
    """paged_gqa_attn on a bf16 q quantised inside the call to e4m3 with one per-tensor scale."""
    lib = load()
    d = _pack(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, out)
    _check(lib.paged_gqa_attn_quant_q(*d[:6], float(k_descale), float(v_descale), float(softmax_scale), d[6],
                                      _stream(stream)))


def paged_gqa_sparse_attn(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, indices,
                          k_descale: float, v_descale: float, softmax_scale: float, out, stream=None) -> None:
    """Sparse paged GQA attention: row (t, h) attends the listed positions indices[t, h // G]."""
    lib = load()
    d = _pack(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, indices, out)
    _check(lib.paged_gqa_sparse_attn(*d[:7], float(k_descale), float(v_descale), float(softmax_scale), d[7],
                                     _stream(stream)))


def paged_gqa_cache_write(k_new, v_new, k_cache, v_cache, block_table, seq_lens, query_start_loc,
                          k_descale: float, v_descale: float, stream=None) -> None:
    """Write the new tokens' K and V (bf16 [T, Hkv, 256]) into the e4m3 paged caches."""
    lib = load()
    d = _pack(k_new, v_new, k_cache, v_cache, block_table, seq_lens, query_start_loc)
    _check(lib.paged_gqa_cache_write(*d, float(k_descale), float(v_descale), _stream(stream)))


def _on_device(*tensors) -> None:
    """The tensors are on the current CUDA device (the library launches there)."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != cur:  # (-1 on the CPU)
            raise ValueError(f"every tensor must be on the current CUDA device (cuda:{cur}), got one on {t.device}")


def _workspace(workspace):
    """(address, bytes) of a workspace tensor."""
    if workspace is None:
        return None, 0
    _on_device(workspace)
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return workspace.data_ptr() or None, workspace.numel() * workspace.element_size()


def _pack_fp4(first_cache: int, *tensors):
    """_pack with tensors[first_cache] and the next one as 4-bit caches (uint8 rows of 144 bytes)."""
    for t in tensors[first_cache:first_cache + 2]:
        if t.dtype is not torch.uint8:
            raise ValueError(f"4-bit caches are uint8 tensors, got {t.dtype}")
    return _pack(*tensors, dtypes=_DTYPES_FP4)


def paged_gqa_cache_write_fp4(k_new, v_new, k_cache, v_cache, block_table, seq_lens, query_start_loc,
                              k_descale: float, v_descale: float, stream=None) -> None:
    """Write the new tokens' K and V (bf16 [T, Hkv, 256]) into 4-bit caches (uint8 [NB, Hkv, P, 144])."""
    lib = load()
    _on_device(k_new, v_new, k_cache, v_cache, block_table, seq_lens, query_start_loc)
    d = _pack_fp4(2, k_new, v_new, k_cache, v_cache, block_table, seq_lens, query_start_loc)
    _check(lib.paged_gqa_cache_write_fp4(*d, float(k_descale), float(v_descale), _stream(stream)))


def paged_gqa_cache_read_fp4(k_cache, v_cache, block_table, seq_lens, query_start_loc, k_descale: float,
                             v_descale: float, k_out, v_out, stream=None) -> None:
    """The values 4-bit caches hold for the last tokens of each sequence, as bf16 [T, Hkv, 256]."""
    lib = load()
    _on_device(k_cache, v_cache, block_table, seq_lens, query_start_loc, k_out, v_out)
    d = _pack_fp4(0, k_cache, v_cache, block_table, seq_lens, query_start_loc, k_out, v_out)
    _check(lib.paged_gqa_cache_read_fp4(*d[:5], float(k_descale), float(v_descale), d[5], d[6], _stream(stream)))


def paged_gqa_attn_fp4(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, k_descale: float,
                       v_descale: float, softmax_scale: float, out, stream=None) -> None:
    """paged_gqa_attn on 4-bit caches (uint8 [NB, Hkv, P, 144]); q and out are bf16."""
    lib = load()
    _on_device(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, out)
    d = _pack_fp4(1, q, k_cache, v_cache, block_table, seq_lens, query_start_loc, out)
    _check(lib.paged_gqa_attn_fp4(*d[:6], float(k_descale), float(v_descale), float(softmax_scale), d[6],
                                  _stream(stream)))


def paged_gqa_attn_fp4_ex(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, k_descale: float,
                          v_descale: float, softmax_scale: float, out, workspace, stream=None) -> None:
    """paged_gqa_attn_fp4 with a caller-owned workspace tensor (for stream capture)."""
    lib = load()
    _on_device(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, out)
    d = _pack_fp4(1, q, k_cache, v_cache, block_table, seq_lens, query_start_loc, out)
    _check(lib.paged_gqa_attn_fp4_ex(*d[:6], float(k_descale), float(v_descale), float(softmax_scale), d[6],
                                     *_workspace(workspace), _stream(stream)))


def paged_gqa_rope(q, k, positions, inv_freq, sections, q_out=None, k_out=None, interleaved: bool = False,
                   adjacent: bool = False, stream=None) -> None:
    """Rotary positions [A, T] for q and k (bf16 [T, H, 256]), in place where no output is given.

    sections: A counts that add up to inv_freq's length (float32 [R / 2])."""
    lib = load()
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    _on_device(q, k, positions, inv_freq, q_out, k_out)
    if len(sections) != positions.shape[0]:
        raise ValueError(f"{len(sections)} sections for {positions.shape[0]} axes")
    d = _pack(q, k, positions, inv_freq, q_out, k_out)
    _check(lib.paged_gqa_rope(*d[:4], (ctypes.c_int32 * len(sections))(*sections), int(interleaved), int(adjacent),
                              d[4], d[5], _stream(stream)))


def paged_gqa_build_tables(q_lens, ctx_lens, rows, page_size: int, pages, page_counts, free_pages, num_free, block_table,
                           seq_lens, query_start_loc, slot_map, page_counts_out=None, num_free_out=None,
                           stream=None) -> None:
    """Block table, seq_lens, query_start_loc and slots of a step, from its requests' lengths (int32 tensors).

    page_counts and num_free are updated in place where no output is given."""
    lib = load()
    t = (q_lens, ctx_lens, rows, pages, page_counts, free_pages, num_free, block_table, seq_lens, query_start_loc, slot_map)
    t += tuple(x for x in (page_counts_out, num_free_out) if x is not None)
    _on_device(*t)
    d = _pack(*t)
    counts_out, num_out = d[4] if page_counts_out is None else d[11], d[6] if num_free_out is None else d[-1]
    _check(lib.paged_gqa_build_tables(*d[:3], int(page_size), *d[3:11], counts_out, num_out, _stream(stream)))


def paged_gqa_tree_masks(parents, seq_lens, query_start_loc, masks, positions, stream=None) -> None:
    """Ancestor masks (int32 [T, words]) and positions (int32 [A, T]) of token trees from their parents."""
    lib = load()
    _on_device(parents, seq_lens, query_start_loc, masks, positions)
    d = _pack(parents, seq_lens, query_start_loc, masks, positions)
    _check(lib.paged_gqa_tree_masks(*d, _stream(stream)))


def paged_gqa_attn_tree(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, masks, k_descale: float,
                        v_descale: float, softmax_scale: float, out, stream=None) -> None:
    """paged_gqa_attn where the new tokens see each other by masks (int32 [T, words]); q is bf16."""
    lib = load()
    _on_device(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, masks, out)
    d = _pack(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, masks, out)
    _check(lib.paged_gqa_attn_tree(*d[:7], float(k_descale), float(v_descale), float(softmax_scale), d[7],
                                   _stream(stream)))


def paged_gqa_attn_tree_ex(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, masks, k_descale: float,
                           v_descale: float, softmax_scale: float, out, workspace, stream=None) -> None:
    """paged_gqa_attn_tree with a caller-owned workspace tensor (for stream capture)."""
    lib = load()
    _on_device(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, masks, out)
    d = _pack(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, masks, out)
    _check(lib.paged_gqa_attn_tree_ex(*d[:7], float(k_descale), float(v_descale), float(softmax_scale), d[7],
                                      *_workspace(workspace), _stream(stream)))


def paged_gqa_cache_keep(k_cache, v_cache, block_table, seq_lens, query_start_loc, kept, num_kept, seq_lens_out,
                         stream=None) -> None:
    """Move the accepted new tokens' K and V (kept: int32 [S, D], num_kept of them) right behind the context."""
    lib = load()
    _on_device(k_cache, v_cache, block_table, seq_lens, query_start_loc, kept, num_kept, seq_lens_out)
    d = _pack(k_cache, v_cache, block_table, seq_lens, query_start_loc, kept, num_kept, seq_lens_out)
    _check(lib.paged_gqa_cache_keep(*d, _stream(stream)))


def paged_gqa_attn_prompt(q, k, v, query_start_loc, softmax_scale: float, out, lse=None, stream=None) -> None:
    """Causal attention over whole packed prompts: q [T, Hq, 256], k and v [T, Hkv, 256] in bf16 or f16."""
    lib = load()
    t = (q, k, v, query_start_loc, out) + (() if lse is None else (lse,))
    _on_device(*t)
    d = _pack(*t)
    _check(lib.paged_gqa_attn_prompt(*d[:4], float(softmax_scale), d[4], d[5] if lse is not None else None,
                                     _stream(stream)))


def paged_gqa_attn_prompt_ex(q, k, v, query_start_loc, softmax_scale: float, out, lse, workspace, stream=None) -> None:
    """paged_gqa_attn_prompt with a caller-owned workspace tensor (for stream capture); lse may be None."""
    lib = load()
    t = (q, k, v, query_start_loc, out) + (() if lse is None else (lse,))
    _on_device(*t)
    d = _pack(*t)
    _check(lib.paged_gqa_attn_prompt_ex(*d[:4], float(softmax_scale), d[4], d[5] if lse is not None else None,
                                        *_workspace(workspace), _stream(stream)))


def paged_gqa_prompt_workspace_size(num_seqs: int, total_tokens: int, num_q_heads: int, num_kv_heads: int, device: int = 0) -> int:
    return int(load().paged_gqa_prompt_workspace_size(num_seqs, total_tokens, num_q_heads, num_kv_heads, device))


def paged_gqa_workspace_size(num_seqs: int, total_q: int, num_q_heads: int, num_kv_heads: int,
                             page_size: int, max_blocks_per_seq: int, device: int = 0) -> int:
    return int(load().paged_gqa_workspace_size(num_seqs, total_q, num_q_heads, num_kv_heads, page_size,
                                               max_blocks_per_seq, device))


def paged_gqa_last_error() -> str:
    return load().paged_gqa_last_error().decode(errors="replace")


def paged_gqa_check_device_errors(stream=None) -> int:
    """Synchronise, read and clear the device error word; returns the status code."""
    return int(load().paged_gqa_check_device_errors(_stream(stream)))


def paged_gqa_set_path(path: int) -> int:
    r = int(load().paged_gqa_set_path(path))
    if r < 0:
        _check(r)
    return r


def paged_gqa_set_stall_test(wait_ns: int) -> int:
    """Failure-path test hook: tcgen05 CTAs first wait wait_ns on a barrier nothing
    arrives on (0 turns it off). Returns the previous value."""
    return int(load().paged_gqa_set_stall_test(int(wait_ns)))


def paged_gqa_last_plan() -> dict:
    buf = (ctypes.c_int64 * 8)()
    _check(load().paged_gqa_last_plan(buf))
    keys = ("verify_ctas", "prefill_ctas", "kernels_launched", "path_bits", "max_verify_blocks",
            "max_prefill_blocks", "workspace_bytes", "verify_self_planned")
    return dict(zip(keys, list(buf)))


def paged_gqa_set_kernel_events(cls: int, start=None, stop=None) -> None:
    """Record torch.cuda.Event pairs around the class-`cls` attention kernel (None clears)."""
    for e in (start, stop):
        if e is not None and not e.cuda_event:
            e.record()  # torch creates the CUDA event lazily, on first record
    h0 = start.cuda_event if start is not None else None
    h1 = stop.cuda_event if stop is not None else None
    _check(load().paged_gqa_set_kernel_events(int(cls), h0, h1))


def paged_gqa_version() -> int:
    return int(load().paged_gqa_version())
