"""Pages of the paged cache that are shared, copied, given back and moved, on CUDA tensors.

``fork_block_tables``     a new batch's rows from rows of the old one, their pages shared
``compact_block_tables``  the highest pages in use into the lowest free ones
``copy_pages``            the copies that either names, in the caches of all layers

As the operators of ``step``: argument marshalling for the C ABI (through the compiled calls where
they are built), on the current stream of the tensors' device (or ``stream``), and a call can be
captured in a CUDA graph.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence

import torch

from . import step
from .step import _call, _empty, _I32, _index, _ints, _refuse_ints, _sizes

_p, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class PaPageTensor(ctypes.Structure):
    _fields_ = [("data", _p), ("page_bytes", _i64)]


class ForkedTables(NamedTuple):
    """The new batch, the copies that its rows need first, and the page allocator's next state."""
    past_seqlens: torch.Tensor  # (new_batch,)
    blocks_held: torch.Tensor   # (new_batch,)
    block_table: torch.Tensor   # (new_batch, columns)
    copies: torch.Tensor        # (new_batch, 2): from, to; -1 behind the last
    free_state: torch.Tensor    # (2,): head, count
    error: torch.Tensor         # (1,): 0, or why the fork was refused


class CompactedTables(NamedTuple):
    """The renamed table, the moves to make before it is used, and the page allocator's next state."""
    block_table: torch.Tensor   # (B, columns)
    copies: torch.Tensor        # (max_moves, 2): from, to; -1 behind the last
    free_state: torch.Tensor    # (2,): 0, count
    pages_end: torch.Tensor     # (1,): one more than the highest page in use
    error: torch.Tensor         # (1,): 0, or why nothing was moved


_bound = None


def _library():
    global _bound
    if _bound is None:
        lib = step._library()
        size = ctypes.c_size_t
        lib.pa_pool_workspace_size.argtypes = [_i32]
        lib.pa_pool_workspace_size.restype = size
        lib.pa_fork_block_tables.argtypes = [_p] * 7 + [_i32] * 6 + [_p] * 7 + [size, _p]
        lib.pa_compact_block_tables.argtypes = [_p] * 4 + [_i32] * 5 + [_p] * 6 + [size, _p]
        lib.pa_copy_pages.argtypes = [ctypes.POINTER(PaPageTensor), _i32, _i32, _p, _i32, _p, _p]
        for f in (lib.pa_fork_block_tables, lib.pa_compact_block_tables, lib.pa_copy_pages):
            f.restype = ctypes.c_int
        _bound = lib
    return _bound


def pool_workspace_size(num_blocks: int) -> int:
    """Bytes of the workspace of fork_block_tables and compact_block_tables (pa_pool_workspace_size)."""
    _sizes(num_blocks=num_blocks)
    return int(_library().pa_pool_workspace_size(num_blocks))


def _workspace(workspace, size, index, device, stream):
    """The caller's workspace, or one of the call's own."""
    if workspace is None:
        return _empty(max(size, 16), torch.uint8, device, stream)
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{index}")
    return workspace


def _check_pinned(pinned, num_blocks, index):
    if pinned is None:
        return None
    if pinned.dtype not in (torch.bool, torch.uint8):
        raise TypeError("pinned must be bool or uint8")
    if pinned.get_device() != index or pinned.shape != (num_blocks,) or not pinned.is_contiguous():
        raise ValueError(f"pinned must be a contiguous (num_blocks,) tensor on cuda:{index}")
    return pinned.data_ptr()


def _check_out(out, index, shapes):
    for name, t, shape in zip(out._fields, out, shapes):
        _refuse_ints(index, **{"out." + name: t})
        if t.shape != shape:
            raise ValueError(f"out.{name} must be {shape}")


def fork_block_tables(parents: torch.Tensor, past_seqlens: torch.Tensor, blocks_held: torch.Tensor,
                      block_table: torch.Tensor, free_blocks: torch.Tensor, free_state: torch.Tensor, *,
                      block_size: int, num_blocks: int, pinned: Optional[torch.Tensor] = None,
                      out: Optional[ForkedTables] = None, workspace: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> ForkedTables:
    """The rows of a new batch from rows of the old one (pa_fork_block_tables).

    ``parents`` (new_batch,): for each new row the old row that it continues, any of them any
    number of times, or -1 for an empty row. Rows share their parent's whole pages; the last page,
    where it is partly filled, stays with one row and every other one gets a page from the ring
    ``free_blocks`` (``free_state`` = [head, count]) and an entry (old page, new page) in
    ``copies``: call ``copy_pages`` with it before the next cache write. Pages that no row holds
    any more go back to the ring, which is updated in place. ``pinned`` (num_blocks,) marks pages
    that something else holds too: not given back, not written to. ``out``: a ForkedTables to
    write to, in memory other than the old batch's. A fork that cannot be served changes nothing,
    describes empty rows and says why in ``error``. A request that shares pages is ended by a -1
    here; ``build_block_tables`` gives every page of a finished request back, shared or not."""
    if out is None and workspace is None and stream is None:
        made = (step._fast or step._load_fast()).fork_block_tables(parents, past_seqlens, blocks_held, block_table,
                                                                   free_blocks, free_state, pinned, block_size, num_blocks)
        if made is not None:
            return ForkedTables._make(made)
    index = _index(block_table, "block_table")
    if not _ints(index, parents, past_seqlens, blocks_held, block_table, free_blocks, free_state):
        _refuse_ints(index, parents=parents, past_seqlens=past_seqlens, blocks_held=blocks_held,
                     block_table=block_table, free_blocks=free_blocks, free_state=free_state)
    shape, table = past_seqlens.shape, block_table.shape
    if (len(shape) != 1 or blocks_held.shape != shape or len(table) != 2 or table[0] != shape[0] or parents.dim() != 1 or
            free_blocks.dim() != 1 or free_state.shape != (2,)):
        raise ValueError("past_seqlens and blocks_held must be (B,), block_table (B, columns), parents and free_blocks "
                         "1-D and free_state (2,)")
    B, columns = table
    n, cap = parents.shape[0], free_blocks.shape[0]
    _sizes(requests=B, new_requests=n, columns=columns, block_size=block_size, num_blocks=num_blocks, free_blocks=cap)
    pins = _check_pinned(pinned, num_blocks, index)
    shapes = ((n,), (n,), (n, columns), (n, 2), (2,), (1,))
    if out is None:
        # one allocation; the copies' pairs first, which are aligned to 8 bytes
        parts = torch.unsafe_split_with_sizes(_empty(n * (columns + 4) + 3, _I32, block_table.device, stream),
                                              (2 * n, n * columns, n, n, 2, 1))
        out = ForkedTables(parts[2], parts[3], parts[1].view(n, columns), parts[0].view(n, 2), parts[4], parts[5])
    else:
        _check_out(out, index, shapes)
    lib = _library()
    ws = _workspace(workspace, lib.pa_pool_workspace_size(num_blocks), index, block_table.device, stream)
    past_out, held_out, table_out, copies, state_out, error = out
    _call("pa_fork_block_tables", index, stream, lib.pa_fork_block_tables, parents.data_ptr(), past_seqlens.data_ptr(),
          blocks_held.data_ptr(), block_table.data_ptr(), free_blocks.data_ptr(), free_state.data_ptr(), pins, B, n,
          columns, block_size, num_blocks, cap, past_out.data_ptr(), held_out.data_ptr(), table_out.data_ptr(),
          copies.data_ptr(), state_out.data_ptr(), error.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return out


def compact_block_tables(blocks_held: torch.Tensor, block_table: torch.Tensor, free_blocks: torch.Tensor, *,
                         num_blocks: int, max_moves: int, pinned: Optional[torch.Tensor] = None,
                         out: Optional[CompactedTables] = None, workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> CompactedTables:
    """Moves up to ``max_moves`` of the highest pages in use into the lowest free ones
    (pa_compact_block_tables). In use are the first ``blocks_held`` entries of the rows and the
    ``pinned`` pages (bool (num_blocks,)), which stay where they are; everything else is taken to
    be free. Returns the renamed table and the moves, which ``copy_pages`` makes before the table
    is used; the ring ``free_blocks`` is rebuilt in place from all free pages in ascending order.
    From ``pages_end`` on the pool is free. ``out``: a CompactedTables to write to; its
    ``block_table`` may be ``block_table`` itself."""
    if out is None and workspace is None and stream is None:
        made = (step._fast or step._load_fast()).compact_block_tables(blocks_held, block_table, free_blocks, pinned,
                                                                      num_blocks, max_moves)
        if made is not None:
            return CompactedTables._make(made)
    index = _index(block_table, "block_table")
    if not _ints(index, blocks_held, block_table, free_blocks):
        _refuse_ints(index, blocks_held=blocks_held, block_table=block_table, free_blocks=free_blocks)
    table = block_table.shape
    if len(table) != 2 or blocks_held.shape != table[:1] or free_blocks.dim() != 1:
        raise ValueError("blocks_held must be (B,), block_table (B, columns) and free_blocks 1-D")
    B, columns = table
    cap = free_blocks.shape[0]
    _sizes(requests=B, columns=columns, num_blocks=num_blocks, max_moves=max_moves, free_blocks=cap)
    pins = _check_pinned(pinned, num_blocks, index)
    if out is None:
        if max_moves < 0:
            raise ValueError("max_moves must not be negative")
        parts = torch.unsafe_split_with_sizes(_empty(2 * max_moves + B * columns + 4, _I32, block_table.device, stream),
                                              (2 * max_moves, B * columns, 2, 1, 1))
        out = CompactedTables(parts[1].view(B, columns), parts[0].view(max_moves, 2), *parts[2:])
    else:
        _check_out(out, index, ((B, columns), (max_moves, 2), (2,), (1,), (1,)))
    lib = _library()
    ws = _workspace(workspace, lib.pa_pool_workspace_size(num_blocks), index, block_table.device, stream)
    table_out, copies, state_out, end, error = out
    _call("pa_compact_block_tables", index, stream, lib.pa_compact_block_tables, blocks_held.data_ptr(),
          block_table.data_ptr(), free_blocks.data_ptr(), pins, B, columns, num_blocks, cap, max_moves,
          table_out.data_ptr(), copies.data_ptr(), state_out.data_ptr(), end.data_ptr(), error.data_ptr(),
          ws.data_ptr(), ws.numel() * ws.element_size())
    return out


def copy_pages(tensors: Sequence[torch.Tensor], copies: torch.Tensor, *, error: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> None:
    """Page ``copies[i][1]`` of every tensor becomes a copy of its page ``copies[i][0]``
    (pa_copy_pages), entries of -1 passed over. ``tensors``: up to 256 contiguous tensors whose
    first extent counts the same pages, of any type: the key and value caches of all layers, page
    bounds. A page may be the target of one entry only, and then the source of none."""
    if stream is None and (step._fast or step._load_fast()).copy_pages(tensors, copies, error):
        return
    if not len(tensors):
        return
    index = _index(copies, "copies")
    if not _ints(index, copies):
        _refuse_ints(index, copies=copies)
    if copies.dim() != 2 or copies.shape[1] != 2:
        raise ValueError("copies must be (entries, 2)")
    num_blocks = tensors[0].shape[0] if tensors[0].dim() else 0
    _sizes(tensors=len(tensors), num_blocks=num_blocks, copies=copies.shape[0])
    pages = (PaPageTensor * len(tensors))()
    for i, t in enumerate(tensors):
        if t.get_device() != index or not t.is_contiguous() or t.dim() == 0 or t.shape[0] != num_blocks:
            raise ValueError(f"tensors must be contiguous (num_blocks, ...) tensors of the same pages on cuda:{index}")
        pages[i].data = t.data_ptr()
        pages[i].page_bytes = t.numel() // num_blocks * t.element_size() if num_blocks else 16
    if error is not None:
        if not _ints(index, error):
            _refuse_ints(index, error=error)
        if error.numel() != 1:
            raise ValueError("error must have one element")
    _call("pa_copy_pages", index, stream, _library().pa_copy_pages, pages, len(tensors), num_blocks, copies.data_ptr(),
          copies.shape[0], None if error is None else error.data_ptr())
