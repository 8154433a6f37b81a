"""The operators of a serving step around the attention call, on CUDA tensors.

``build_block_tables``      prefix sums, positions, slots and block tables from the requests' lengths
``qk_norm_rope``            RMSNorm and rotary embedding of query and key rows
``update_page_bounds``      per-page bounds of the keys a step has cached
``select_pages``            the pages each query row attends, by a score against the bounds
``sparse_paged_attention``  attention over the selected pages

As ``paged_attention``: argument marshalling only, for the C ABI of ``libpagedattn.so``; the
work runs on the current stream of the tensors' device (or ``stream``), and a call can be
captured in a CUDA graph. An int32 tensor of one element passed as ``error`` collects the
``DEVERR_*`` bits of problems that only device data reveals.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

_I32 = torch.int32
_p, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class PaSparseDims(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "num_tokens", "batch_size", "num_heads", "kv_num_heads", "head_size", "num_blocks", "block_size",
        "max_blocks_per_sequence", "dtype", "top_k", "query_block", "sink_pages", "local_pages", "reserved")] + [
            ("query_stride", _i64)]


class BlockTables(NamedTuple):
    """What a step's attention call takes, and the page allocator's next state."""
    cumulative_sequence_length: torch.Tensor  # (B + 1,)
    slot_mapping: torch.Tensor                # (num_tokens,)
    positions: torch.Tensor                   # (num_tokens,)
    blocks_held: torch.Tensor                 # (B,)
    free_state: torch.Tensor                  # (2,): head, count
    error: torch.Tensor                       # (1,): 0, or why the step was refused


_bound = None


def _library():
    global _bound
    if _bound is None:
        from . import PaQkPrep, load_library
        lib = load_library()
        dims = ctypes.POINTER(PaSparseDims)
        lib.pa_build_block_tables.argtypes = [_p] * 6 + [_i32] * 5 + [_p] * 7
        lib.pa_qk_norm_rope.argtypes = [_p, _p, _p, ctypes.POINTER(PaQkPrep)] + [_i32] * 6 + [_i64, _i64, _p, _p, _i64,
                                                                                              _i64, _p]
        lib.pa_update_page_bounds.argtypes = [_p] * 6 + [dims, _p, _p]
        lib.pa_select_pages.argtypes = [_p] * 6 + [dims, _p, _p, _p]
        lib.pa_sparse_paged_attention.argtypes = [_p] * 7 + [_f32, _p, _p, dims, _p, _p]
        for f in (lib.pa_build_block_tables, lib.pa_qk_norm_rope, lib.pa_update_page_bounds, lib.pa_select_pages,
                  lib.pa_sparse_paged_attention):
            f.restype = ctypes.c_int
        _bound = lib
    return _bound


@functools.lru_cache(maxsize=256)
def _dims(*v) -> PaSparseDims:
    return PaSparseDims(*v)


def _check_int32(device, **tensors):
    for name, t in tensors.items():
        if t.dtype != _I32:
            raise TypeError(f"{name} must be int32")
        if t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor on {device}")


def _check_cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _rows(t, name, width, dtype, device):
    """The row stride of a 2-D tensor whose rows are contiguous (it may be a view of wider rows)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.device != device or t.dim() != 2 or t.shape[1] != width or (width > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be (rows, {width}) on {device} with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else -(-max(width, t.stride(0)) // 8) * 8


def _call(where, device, stream, function, *args):
    """Calls function(*args, stream) with the tensors' device current."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(where, device, stream, function, *args)
    status = function(*args, (stream or torch.cuda.current_stream(device)).cuda_stream)
    if status:
        from . import PagedAttentionError
        raise PagedAttentionError(status, where)


def build_block_tables(past_seqlens: torch.Tensor, query_lens: torch.Tensor, blocks_held: torch.Tensor,
                       block_table: torch.Tensor, free_blocks: torch.Tensor, free_state: torch.Tensor, *,
                       block_size: int, num_tokens: int, out: Optional[BlockTables] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> BlockTables:
    """One step's batch description from the requests' lengths (pa_build_block_tables).

    ``query_lens`` (B): new rows of each request, 0 for none, -1 for a finished request, whose
    pages go back. ``blocks_held`` (B): pages each request holds. ``block_table`` (B, columns)
    and ``free_blocks`` (a ring of page numbers with ``free_state`` = [head, count]) are updated
    in place; the new ``blocks_held`` and ``free_state`` are returned, with the arguments of the
    attention call for ``num_tokens`` rows (those behind the last request have slot and position
    -1). ``out``: a BlockTables to write to, as a captured step keeps it. A step that cannot be
    served changes nothing, describes an empty batch and says why in ``error``."""
    device = _check_cuda(block_table, "block_table")
    _check_int32(device, past_seqlens=past_seqlens, query_lens=query_lens, blocks_held=blocks_held,
                 block_table=block_table, free_blocks=free_blocks, free_state=free_state)
    B = past_seqlens.shape[0]
    if (past_seqlens.dim() != 1 or query_lens.shape != past_seqlens.shape or blocks_held.shape != past_seqlens.shape or
            block_table.dim() != 2 or block_table.shape[0] != B or free_blocks.dim() != 1 or free_state.shape != (2,)):
        raise ValueError("past_seqlens, query_lens and blocks_held must be (B,), block_table (B, columns), "
                         "free_blocks 1-D and free_state (2,)")
    sizes = (B + 1, num_tokens, num_tokens, B, 2, 1)
    if out is None:
        if num_tokens < 0:
            raise ValueError("num_tokens must not be negative")
        out = BlockTables._make(torch.empty(sum(sizes), dtype=_I32, device=device).split(sizes))
    else:
        for name, t, n in zip(BlockTables._fields, out, sizes):
            _check_int32(device, **{"out." + name: t})
            if t.shape != (n,):
                raise ValueError(f"out.{name} must have {n} elements")
    _call("pa_build_block_tables", device, stream, _library().pa_build_block_tables,
          past_seqlens.data_ptr(), query_lens.data_ptr(), blocks_held.data_ptr(), block_table.data_ptr(),
          free_blocks.data_ptr(), free_state.data_ptr(), B, num_tokens, block_table.shape[1], block_size,
          free_blocks.shape[0], *[t.data_ptr() for t in out])
    return out


def qk_norm_rope(query: torch.Tensor, key: torch.Tensor, positions: torch.Tensor, *, num_heads: int,
                 kv_num_heads: int, q_norm_weight: Optional[torch.Tensor] = None,
                 k_norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, rotary_dim: int = 0,
                 theta: float = 10000.0, interleaved: bool = False, query_out: Optional[torch.Tensor] = None,
                 key_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """RMSNorm of every query and key head (with a weight), then the rotary embedding at
    ``positions`` (N,), rounded once (pa_qk_norm_rope). ``query`` (N, num_heads * head_size) and
    ``key`` (N, kv_num_heads * head_size) may be views of packed rows; ``query_out`` / ``key_out``
    may be ``query`` / ``key`` themselves. Rows with a negative position are left as they were.
    ``interleaved`` pairs components 2u and 2u + 1 instead of u and u + rotary_dim / 2. Returns
    (query_out, key_out)."""
    from . import PaQkPrep, _DTYPES
    device, dtype = _check_cuda(query, "query"), query.dtype
    if dtype not in _DTYPES:
        raise TypeError("query must be float16 or bfloat16")
    if num_heads <= 0 or kv_num_heads <= 0 or query.dim() != 2 or query.shape[1] % num_heads:
        raise ValueError("query must be (rows, num_heads * head_size)")
    N, head_size = query.shape[0], query.shape[1] // num_heads
    qw, kw = num_heads * head_size, kv_num_heads * head_size
    qs, ks = _rows(query, "query", qw, dtype, device), _rows(key, "key", kw, dtype, device)
    if query_out is None:
        query_out = torch.empty((N, qw), dtype=dtype, device=device)
        qos = qw
    else:
        qos = _rows(query_out, "query_out", qw, dtype, device)
    if key_out is None:
        key_out = torch.empty((N, kw), dtype=dtype, device=device)
        kos = kw
    else:
        kos = _rows(key_out, "key_out", kw, dtype, device)
    _check_int32(device, positions=positions)
    if positions.shape != (N,) or key.shape[0] != N or query_out.shape[0] != N or key_out.shape[0] != N:
        raise ValueError("query, key, positions and the outputs must have the same number of rows")
    for name, w in (("q_norm_weight", q_norm_weight), ("k_norm_weight", k_norm_weight)):
        if w is not None and (w.dtype != dtype or w.device != device or w.shape != (head_size,) or
                              not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous tensor of head_size values of the query dtype")
    prep = PaQkPrep(None if q_norm_weight is None else q_norm_weight.data_ptr(),
                    None if k_norm_weight is None else k_norm_weight.data_ptr(), eps, theta, rotary_dim, 0)
    _call("pa_qk_norm_rope", device, stream, _library().pa_qk_norm_rope, query.data_ptr(), key.data_ptr(),
          positions.data_ptr(), prep, int(interleaved), N, num_heads, kv_num_heads, head_size, _DTYPES[dtype],
          qs, ks, query_out.data_ptr(), key_out.data_ptr(), qos, kos)
    return query_out, key_out


def _batch(device, cum, past, block_table, error):
    _check_int32(device, cumulative_sequence_length=cum, past_seqlens=past, block_table=block_table)
    B = past.shape[0]
    if past.dim() != 1 or cum.shape != (B + 1,) or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("cumulative_sequence_length must have batch_size + 1 entries, block_table batch_size rows")
    if error is None:
        return B, None
    _check_int32(device, error=error)
    if error.numel() != 1:
        raise ValueError("error must have one element")
    return B, error.data_ptr()


def _check_bounds(device, page_bounds, bound_scale, kv_num_heads):
    if page_bounds.dtype != torch.int8 or bound_scale.dtype != torch.float32:
        raise TypeError("page_bounds must be int8 and bound_scale float32")
    if (page_bounds.dim() != 4 or page_bounds.shape[1] != kv_num_heads or page_bounds.shape[2] != 2 or
            bound_scale.shape != (kv_num_heads, page_bounds.shape[3])):
        raise ValueError("page_bounds must be (num_blocks, kv_num_heads, 2, head_size), bound_scale "
                         "(kv_num_heads, head_size)")
    if (page_bounds.device != device or bound_scale.device != device or not page_bounds.is_contiguous() or
            not bound_scale.is_contiguous()):
        raise ValueError(f"page_bounds and bound_scale must be contiguous tensors on {device}")


def update_page_bounds(key_cache: torch.Tensor, page_bounds: torch.Tensor, bound_scale: torch.Tensor,
                       cumulative_sequence_length: torch.Tensor, past_seqlens: torch.Tensor,
                       block_table: torch.Tensor, *, num_tokens: int, error: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The bounds of the pages that this step's keys are in (pa_update_page_bounds), after the
    cache write. ``page_bounds`` int8 (num_blocks, kv_num_heads, 2, head_size) is updated in place
    and returned: per page, KV head and channel the least and the largest code of the page's keys
    in units of ``bound_scale`` (float32 (kv_num_heads, head_size)). ``num_tokens``: a bound on
    the step's rows, as the shape of its query. For a cache that is there already pass
    ``past_seqlens`` of 0 and the whole lengths."""
    from . import _DTYPES
    device = _check_cuda(key_cache, "key_cache")
    if key_cache.dtype not in _DTYPES:
        raise TypeError("key_cache must be float16 or bfloat16")
    if key_cache.dim() != 4 or not key_cache.is_contiguous():
        raise ValueError("key_cache must be a contiguous (num_blocks, block_size, kv_num_heads, head_size) tensor")
    blocks, bs, kvh, hs = key_cache.shape
    _check_bounds(device, page_bounds, bound_scale, kvh)
    if page_bounds.shape[0] != blocks or page_bounds.shape[3] != hs:
        raise ValueError("page_bounds must have the key cache's pages and head size")
    B, err = _batch(device, cumulative_sequence_length, past_seqlens, block_table, error)
    d = _dims(num_tokens, B, kvh, kvh, hs, blocks, bs, block_table.shape[1], _DTYPES[key_cache.dtype], 1, 1, 0, 1, 0,
              kvh * hs)
    _call("pa_update_page_bounds", device, stream, _library().pa_update_page_bounds, key_cache.data_ptr(),
          page_bounds.data_ptr(), bound_scale.data_ptr(), cumulative_sequence_length.data_ptr(),
          past_seqlens.data_ptr(), block_table.data_ptr(), d, err)
    return page_bounds


def select_pages(query: torch.Tensor, page_bounds: torch.Tensor, bound_scale: torch.Tensor,
                 cumulative_sequence_length: torch.Tensor, past_seqlens: torch.Tensor, block_table: torch.Tensor, *,
                 num_heads: int, kv_num_heads: int, block_size: int, top_k: int, query_block: int = 1,
                 sink_pages: int = 1, local_pages: int = 1, selected: Optional[torch.Tensor] = None,
                 error: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The ``top_k`` pages of its history that each query row attends, per KV head
    (pa_select_pages): int32 (N, kv_num_heads, top_k), logical pages in ascending order, then -1.
    Rows [j R, (j + 1) R) of a sequence, R = ``query_block``, share a selection: the first
    ``sink_pages`` pages, the last ``local_pages`` up to the block's first row, the pages of its
    rows, and the best others by an upper bound of q.k summed over the block's rows and heads,
    in whole numbers. ``query`` (N, num_heads * head_size) may be a view of packed rows."""
    from . import _DTYPES
    device, dtype = _check_cuda(query, "query"), query.dtype
    if dtype not in _DTYPES:
        raise TypeError("query must be float16 or bfloat16")
    _check_bounds(device, page_bounds, bound_scale, kv_num_heads)
    blocks, hs = page_bounds.shape[0], page_bounds.shape[3]
    stride = _rows(query, "query", num_heads * hs, dtype, device)
    B, err = _batch(device, cumulative_sequence_length, past_seqlens, block_table, error)
    N = query.shape[0]
    if selected is None:
        selected = torch.empty((N, kv_num_heads, max(top_k, 0)), dtype=_I32, device=device)
    else:
        _check_int32(device, selected=selected)
        if selected.shape != (N, kv_num_heads, top_k):
            raise ValueError("selected must be (rows, kv_num_heads, top_k)")
    d = _dims(N, B, num_heads, kv_num_heads, hs, blocks, block_size, block_table.shape[1], _DTYPES[dtype], top_k,
              query_block, sink_pages, local_pages, 0, stride)
    _call("pa_select_pages", device, stream, _library().pa_select_pages, query.data_ptr(), page_bounds.data_ptr(),
          bound_scale.data_ptr(), cumulative_sequence_length.data_ptr(), past_seqlens.data_ptr(),
          block_table.data_ptr(), d, selected.data_ptr(), err)
    return selected


def sparse_paged_attention(query: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                           cumulative_sequence_length: torch.Tensor, past_seqlens: torch.Tensor,
                           block_table: torch.Tensor, selected: torch.Tensor, *, num_heads: int, kv_num_heads: int,
                           scale: float = 0.0, query_block: int = 1, output: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None, error: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``paged_attention``'s read path over selected pages only (pa_sparse_paged_attention): each
    row attends the keys up to its own position that lie in the pages ``selected`` for its query
    block. The caches already hold this step's rows. Returns ``output`` (N, num_heads *
    head_size); ``lse`` (float32 (N, num_heads)) receives the rows' log-sum-exp. A row that
    attends nothing gives zeros and -inf; rows behind the last sequence are left as they were."""
    from . import _DTYPES
    device, dtype = _check_cuda(query, "query"), query.dtype
    if dtype not in _DTYPES:
        raise TypeError("query must be float16 or bfloat16")
    for name, t in (("key_cache", key_cache), ("value_cache", value_cache)):
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}")
        if t.device != device or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous (num_blocks, block_size, kv_num_heads, head_size) tensor "
                             f"on {device}")
    blocks, bs, kvh, hs = key_cache.shape
    if kvh != kv_num_heads or value_cache.shape != key_cache.shape:
        raise ValueError("cache shape must be (num_blocks, block_size, kv_num_heads, head_size)")
    stride = _rows(query, "query", num_heads * hs, dtype, device)
    B, err = _batch(device, cumulative_sequence_length, past_seqlens, block_table, error)
    N = query.shape[0]
    _check_int32(device, selected=selected)
    if selected.dim() != 3 or selected.shape[0] != N or selected.shape[1] != kvh:
        raise ValueError("selected must be (rows, kv_num_heads, top_k)")
    if output is None:
        output = torch.empty((N, num_heads * hs), dtype=dtype, device=device)
    elif output.dtype != dtype or output.device != device or output.shape != (N, num_heads * hs) or \
            not output.is_contiguous():
        raise ValueError("output must be contiguous (rows, num_heads * head_size) of the query dtype")
    if lse is not None and (lse.dtype != torch.float32 or lse.device != device or lse.shape != (N, num_heads) or
                            not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 (rows, num_heads)")
    d = _dims(N, B, num_heads, kvh, hs, blocks, bs, block_table.shape[1], _DTYPES[dtype], selected.shape[2],
              query_block, 0, 1, 0, stride)
    _call("pa_sparse_paged_attention", device, stream, _library().pa_sparse_paged_attention, query.data_ptr(),
          key_cache.data_ptr(), value_cache.data_ptr(), cumulative_sequence_length.data_ptr(),
          past_seqlens.data_ptr(), block_table.data_ptr(), selected.data_ptr(), scale, output.data_ptr(),
          None if lse is None else lse.data_ptr(), d, err)
    return output
