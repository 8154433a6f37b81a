"""The operators of a serving step around the attention call, on CUDA tensors.

``build_block_tables``      prefix sums, positions, slots and block tables from the requests' lengths
``qk_norm_rope``            RMSNorm and rotary embedding of query and key rows
``update_page_bounds``      per-page bounds of the keys a step has cached
``select_pages``            the pages each query row attends, by a score against the bounds
``sparse_paged_attention``  attention over the selected pages

As ``paged_attention``: argument marshalling only, for the C ABI of ``libpagedattn.so``. The
common case (outputs of the call's own, the current stream and device) goes through the compiled
``_step_binding`` (where it is built for this torch), whose checks take a microsecond; everything else, refusals
among it, through the code here. The work runs on the current stream of the tensors' device (or ``stream``), and a call can be
captured in a CUDA graph. An int32 tensor of one element passed as ``error`` collects the
``DEVERR_*`` bits of problems that only device data reveals. With ``stream`` the caller orders
that stream after the work that makes the inputs, and other streams after the call.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import warnings
from typing import NamedTuple, Optional

import torch

from .build import binding_path

_I32 = torch.int32
_T = {torch.float16: 0, torch.bfloat16: 1}  # pa_dtype
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


_bound = _prep = None
_fast = None  # the compiled binding, once loaded


class _Absent:
    """Stands in for the compiled calls where they are not built: every call is made in Python."""

    def __getattr__(self, name):
        return lambda *a: None


def _load_fast():
    """The compiled calls (csrc/binding.cpp), given the library's entry points."""
    global _fast
    if _fast is None:
        lib = _library()
        path = binding_path(os.path.dirname(os.path.abspath(__file__)))
        try:
            loader = importlib.machinery.ExtensionFileLoader("_step_binding", path)
            module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_step_binding", loader))
        except ImportError as e:
            warnings.warn(f"no compiled calls, each call takes some microseconds longer: {e} "
                          "(varlen_paged_kv_gb300.build.build() builds them)", RuntimeWarning)
            _fast = _Absent()
            return _fast
        module.bind(*[ctypes.cast(f, _p).value for f in (
            lib.pa_build_block_tables, lib.pa_qk_norm_rope, lib.pa_update_page_bounds, lib.pa_select_pages,
            lib.pa_sparse_paged_attention)])
        from .biased import _library as biased_library
        from .pool import _library as pool_library
        pool_library(), biased_library()
        module.bind_pool(*[ctypes.cast(f, _p).value for f in (
            lib.pa_fork_block_tables, lib.pa_compact_block_tables, lib.pa_copy_pages, lib.pa_biased_paged_attention,
            lib.pa_pool_workspace_size, lib.pa_biased_workspace_size)])
        _fast = module
    return _fast


def _library():
    global _bound
    if _bound is None:
        from . import PaQkPrep, load_library
        global _prep
        lib, _prep = load_library(), PaQkPrep
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


def _sizes(**sizes):
    """Refuses what the C ABI's 32-bit fields cannot hold (ctypes would keep the low bits)."""
    for name, v in sizes.items():
        if not -(1 << 31) <= v < 1 << 31:
            raise ValueError(f"{name} must fit 32 bits")


# (the records hold sizes and scalars only)
@functools.lru_cache(maxsize=256)
def _dims(*v) -> PaSparseDims:
    _sizes(**{n: x for (n, t), x in zip(PaSparseDims._fields_, v) if t is _i32})
    return PaSparseDims(*v)


# The checks run on every call of a serving loop: one pass over the tensors decides, and only a
# call that is refused finds out which of them it was.


def _ints(index, *tensors):
    """Whether all are contiguous int32 tensors on CUDA device ``index``."""
    for t in tensors:
        if t.dtype is not _I32 or t.get_device() != index or not t.is_contiguous():
            return False
    return True


def _refuse_ints(index, **tensors):
    for name, t in tensors.items():
        if t.dtype != _I32:
            raise TypeError(f"{name} must be int32")
        if t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor on cuda:{index}")


def _index(t, name):
    """The CUDA device that the call's tensors are on."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


def _rows(t, name, width, dtype, index):
    """The row stride of a 2-D tensor whose rows are contiguous (it may be a view of wider rows)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    shape, (step, one) = t.shape, t.stride() if t.dim() == 2 else (0, 0)
    if t.get_device() != index or len(shape) != 2 or shape[1] != width or (one != 1 and width > 1):
        raise ValueError(f"{name} must be (rows, {width}) on cuda:{index} with contiguous rows")
    return step if shape[0] > 1 else -(-max(width, step) // 8) * 8


def _empty(shape, dtype, device, stream):
    """A tensor for a kernel of ``stream`` to write: of that stream's memory, so that nothing else
    is still using it, and not given back before work that the current stream has by then."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _call(where, index, stream, function, *args):
    """Calls function(*args, stream) with the tensors' device current; the stream is the caller's
    or that device's current one."""
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _call(where, index, stream, function, *args)
    status = function(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
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
    attention call for ``num_tokens`` rows. Rows behind the last request have slot and position
    -1 and are left alone by the operators here; ``paged_attention`` refuses a batch that ends
    before its rows (DEVERR_BAD_BATCH, nothing written), so where the rows of a captured step are
    a fixed number, a spare request with ``past_seqlens`` 0 takes those left over. ``out``: a BlockTables to write to, as a captured step keeps it. A step that cannot be
    served changes nothing, describes an empty batch and says why in ``error``."""
    if out is None and stream is None:
        made = (_fast or _load_fast()).build_block_tables(past_seqlens, query_lens, blocks_held, block_table, free_blocks,
                                                          free_state, block_size, num_tokens)
        if made is not None:
            return BlockTables._make(made)
    index = _index(block_table, "block_table")
    if not _ints(index, past_seqlens, query_lens, blocks_held, block_table, free_blocks, free_state):
        _refuse_ints(index, past_seqlens=past_seqlens, query_lens=query_lens, blocks_held=blocks_held,
                     block_table=block_table, free_blocks=free_blocks, free_state=free_state)
    shape, table = past_seqlens.shape, block_table.shape
    if (len(shape) != 1 or query_lens.shape != shape or blocks_held.shape != shape or len(table) != 2 or
            table[0] != shape[0] or free_blocks.dim() != 1 or free_state.shape != (2,)):
        raise ValueError("past_seqlens, query_lens and blocks_held must be (B,), block_table (B, columns), "
                         "free_blocks 1-D and free_state (2,)")
    B = shape[0]
    _sizes(requests=B, num_tokens=num_tokens, columns=table[1], block_size=block_size,
           free_blocks=free_blocks.shape[0])
    sizes = (B + 1, num_tokens, num_tokens, B, 2, 1)
    if out is None:
        if num_tokens < 0:
            raise ValueError("num_tokens must not be negative")
        # one allocation; the pieces are tensors of their own
        out = BlockTables._make(torch.unsafe_split_with_sizes(
            _empty(2 * (B + num_tokens + 2), _I32, block_table.device, stream), sizes))
    else:
        for name, t, n in zip(BlockTables._fields, out, sizes):
            _refuse_ints(index, **{"out." + name: t})
            if t.shape != (n,):
                raise ValueError(f"out.{name} must have {n} elements")
    cum, slots, positions, held, state, error = out
    _call("pa_build_block_tables", index, stream, _library().pa_build_block_tables,
          past_seqlens.data_ptr(), query_lens.data_ptr(), blocks_held.data_ptr(), block_table.data_ptr(),
          free_blocks.data_ptr(), free_state.data_ptr(), B, num_tokens, table[1], block_size, free_blocks.shape[0],
          cum.data_ptr(), slots.data_ptr(), positions.data_ptr(), held.data_ptr(), state.data_ptr(), error.data_ptr())
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
    if query_out is None and key_out is None and stream is None:
        made = (_fast or _load_fast()).qk_norm_rope(query, key, positions, num_heads, kv_num_heads, q_norm_weight,
                                                    k_norm_weight, eps, rotary_dim, theta, interleaved)
        if made is not None:
            return made
    index, dtype, shape = _index(query, "query"), query.dtype, query.shape
    if dtype not in _T:
        raise TypeError("query must be float16 or bfloat16")
    if num_heads <= 0 or kv_num_heads <= 0 or len(shape) != 2 or shape[1] % num_heads:
        raise ValueError("query must be (rows, num_heads * head_size)")
    N, qw = shape
    head_size = qw // num_heads
    _sizes(rows=N, num_heads=num_heads, kv_num_heads=kv_num_heads, head_size=head_size, rotary_dim=rotary_dim)
    kw = kv_num_heads * head_size
    qs, ks = _rows(query, "query", qw, dtype, index), _rows(key, "key", kw, dtype, index)
    device = None if query_out is not None and key_out is not None else query.device
    if query_out is None:
        query_out = _empty((N, qw), dtype, device, stream)
        qos = qw
    else:
        qos = _rows(query_out, "query_out", qw, dtype, index)
    if key_out is None:
        key_out = _empty((N, kw), dtype, device, stream)
        kos = kw
    else:
        kos = _rows(key_out, "key_out", kw, dtype, index)
    if not _ints(index, positions):
        _refuse_ints(index, positions=positions)
    if positions.shape != (N,) or key.shape[0] != N or query_out.shape[0] != N or key_out.shape[0] != N:
        raise ValueError("query, key, positions and the outputs must have the same number of rows")
    for name, w in (("q_norm_weight", q_norm_weight), ("k_norm_weight", k_norm_weight)):
        if w is not None and (w.dtype is not dtype or w.get_device() != index or w.shape != (head_size,) or
                              not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous tensor of head_size values of the query dtype")
    lib = _library()
    prep = _prep(None if q_norm_weight is None else q_norm_weight.data_ptr(),
                    None if k_norm_weight is None else k_norm_weight.data_ptr(), eps, theta, rotary_dim, 0)
    _call("pa_qk_norm_rope", index, stream, lib.pa_qk_norm_rope, query.data_ptr(), key.data_ptr(),
          positions.data_ptr(), prep, int(interleaved), N, num_heads, kv_num_heads, head_size, _T[dtype], qs,
          ks, query_out.data_ptr(), key_out.data_ptr(), qos, kos)
    return query_out, key_out


def _batch(index, cum, past, block_table, error):
    if not _ints(index, cum, past, block_table):
        _refuse_ints(index, cumulative_sequence_length=cum, past_seqlens=past, block_table=block_table)
    shape, table = past.shape, block_table.shape
    if len(shape) != 1 or cum.shape != (shape[0] + 1,) or len(table) != 2 or table[0] != shape[0]:
        raise ValueError("cumulative_sequence_length must have batch_size + 1 entries, block_table batch_size rows")
    if error is None:
        return shape[0], table[1], None
    if not _ints(index, error):
        _refuse_ints(index, error=error)
    if error.numel() != 1:
        raise ValueError("error must have one element")
    return shape[0], table[1], error.data_ptr()


def _check_bounds(index, page_bounds, bound_scale, kv_num_heads):
    if page_bounds.dtype is not torch.int8 or bound_scale.dtype is not torch.float32:
        raise TypeError("page_bounds must be int8 and bound_scale float32")
    shape = page_bounds.shape
    if len(shape) != 4 or shape[1] != kv_num_heads or shape[2] != 2 or bound_scale.shape != (kv_num_heads, shape[3]):
        raise ValueError("page_bounds must be (num_blocks, kv_num_heads, 2, head_size), bound_scale "
                         "(kv_num_heads, head_size)")
    if (page_bounds.get_device() != index or bound_scale.get_device() != index or not page_bounds.is_contiguous() or
            not bound_scale.is_contiguous()):
        raise ValueError(f"page_bounds and bound_scale must be contiguous tensors on cuda:{index}")
    return shape[0], shape[3]


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
    if stream is None and (_fast or _load_fast()).update_page_bounds(
            key_cache, page_bounds, bound_scale, cumulative_sequence_length, past_seqlens, block_table, num_tokens,
            error):
        return page_bounds
    index, dtype = _index(key_cache, "key_cache"), key_cache.dtype
    if dtype not in _T:
        raise TypeError("key_cache must be float16 or bfloat16")
    if key_cache.dim() != 4 or not key_cache.is_contiguous():
        raise ValueError("key_cache must be a contiguous (num_blocks, block_size, kv_num_heads, head_size) tensor")
    blocks, bs, kvh, hs = key_cache.shape
    if _check_bounds(index, page_bounds, bound_scale, kvh) != (blocks, hs):
        raise ValueError("page_bounds must have the key cache's pages and head size")
    B, columns, err = _batch(index, cumulative_sequence_length, past_seqlens, block_table, error)
    d = _dims(num_tokens, B, kvh, kvh, hs, blocks, bs, columns, _T[dtype], 1, 1, 0, 1, 0, kvh * hs)
    _call("pa_update_page_bounds", index, stream, _library().pa_update_page_bounds, key_cache.data_ptr(),
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
    rows, and the best others by an estimate from the bounds of the largest q.k, summed over the
    block's rows and heads, in whole numbers. ``query`` (N, num_heads * head_size) may be a view of packed rows."""
    if selected is None and stream is None:
        made = (_fast or _load_fast()).select_pages(
            query, page_bounds, bound_scale, cumulative_sequence_length, past_seqlens, block_table, num_heads,
            kv_num_heads, block_size, top_k, query_block, sink_pages, local_pages, error)
        if made is not None:
            return made
    index, dtype = _index(query, "query"), query.dtype
    if dtype not in _T:
        raise TypeError("query must be float16 or bfloat16")
    blocks, hs = _check_bounds(index, page_bounds, bound_scale, kv_num_heads)
    stride = _rows(query, "query", num_heads * hs, dtype, index)
    B, columns, err = _batch(index, cumulative_sequence_length, past_seqlens, block_table, error)
    N = query.shape[0]
    d = _dims(N, B, num_heads, kv_num_heads, hs, blocks, block_size, columns, _T[dtype], top_k, query_block,
              sink_pages, local_pages, 0, stride)
    if selected is None:
        selected = _empty((N, kv_num_heads, max(top_k, 0)), _I32, query.device, stream)
    else:
        _refuse_ints(index, selected=selected)
        if selected.shape != (N, kv_num_heads, top_k):
            raise ValueError("selected must be (rows, kv_num_heads, top_k)")
    _call("pa_select_pages", index, stream, _library().pa_select_pages, query.data_ptr(), page_bounds.data_ptr(),
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
    attends nothing gives zeros and -inf; rows behind the last sequence are left as they were.
    A pipeline wait that runs out (DEVERR_TIMEOUT, the rows of its block undefined) is told by
    ``error`` only, as there is no workspace to keep it: pass one where that matters."""
    if output is None and stream is None:
        made = (_fast or _load_fast()).sparse_paged_attention(
            query, key_cache, value_cache, cumulative_sequence_length, past_seqlens, block_table, selected, num_heads,
            kv_num_heads, scale, query_block, lse, error)
        if made is not None:
            return made
    index, dtype = _index(query, "query"), query.dtype
    if dtype not in _T:
        raise TypeError("query must be float16 or bfloat16")
    for name, t in (("key_cache", key_cache), ("value_cache", value_cache)):
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}")
        if t.get_device() != index or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous (num_blocks, block_size, kv_num_heads, head_size) tensor "
                             f"on cuda:{index}")
    shape = key_cache.shape
    blocks, bs, kvh, hs = shape
    if kvh != kv_num_heads or value_cache.shape != shape:
        raise ValueError("cache shape must be (num_blocks, block_size, kv_num_heads, head_size)")
    stride = _rows(query, "query", num_heads * hs, dtype, index)
    B, columns, err = _batch(index, cumulative_sequence_length, past_seqlens, block_table, error)
    N = query.shape[0]
    if not _ints(index, selected):
        _refuse_ints(index, selected=selected)
    chosen = selected.shape
    if len(chosen) != 3 or chosen[0] != N or chosen[1] != kvh:
        raise ValueError("selected must be (rows, kv_num_heads, top_k)")
    if output is None:
        output = _empty((N, num_heads * hs), dtype, query.device, stream)
    elif output.dtype is not dtype or output.get_device() != index or output.shape != (N, num_heads * hs) or \
            not output.is_contiguous():
        raise ValueError("output must be contiguous (rows, num_heads * head_size) of the query dtype")
    if lse is not None and (lse.dtype is not torch.float32 or lse.get_device() != index or lse.shape != (N, num_heads) or
                            not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 (rows, num_heads)")
    d = _dims(N, B, num_heads, kvh, hs, blocks, bs, columns, _T[dtype], chosen[2], query_block,
              0, 1, 0, stride)
    _call("pa_sparse_paged_attention", index, stream, _library().pa_sparse_paged_attention, query.data_ptr(),
          key_cache.data_ptr(), value_cache.data_ptr(), cumulative_sequence_length.data_ptr(),
          past_seqlens.data_ptr(), block_table.data_ptr(), selected.data_ptr(), scale, output.data_ptr(),
          None if lse is None else lse.data_ptr(), d, err)
    return output
