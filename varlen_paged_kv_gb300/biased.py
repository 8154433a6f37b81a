"""Attention over the paged cache with capped scores, biases by distance, windows, packed
documents and bidirectional prefixes, on CUDA tensors: argument marshalling for the C ABI."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import step
from .pool import _workspace
from .step import _batch, _call, _empty, _index, _rows, _sizes, _T

_p, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class PaScoreRules(ctypes.Structure):
    _fields_ = [("softcap", _f32), ("window", _i32), ("slopes", _p), ("first_keys", _p), ("prefix_lens", _p),
                ("reserved", _i64)]


class PaBiasedDims(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "num_tokens", "batch_size", "num_heads", "kv_num_heads", "head_size", "num_blocks", "block_size",
        "max_blocks_per_sequence", "dtype", "max_query_len")] + [("query_stride", _i64), ("reserved", _i64)]


_bound = None


def _library():
    global _bound
    if _bound is None:
        lib = step._library()
        lib.pa_biased_workspace_size.argtypes = [_i32]
        lib.pa_biased_workspace_size.restype = ctypes.c_size_t
        lib.pa_biased_paged_attention.argtypes = [_p] * 6 + [_f32, ctypes.POINTER(PaScoreRules), _p, _p,
                                                             ctypes.POINTER(PaBiasedDims), _p, _p, ctypes.c_size_t, _p]
        lib.pa_biased_paged_attention.restype = ctypes.c_int
        _bound = lib
    return _bound


def biased_workspace_size(head_size: int) -> int:
    """Bytes of the workspace of biased_paged_attention (pa_biased_workspace_size)."""
    _sizes(head_size=head_size)
    return int(_library().pa_biased_workspace_size(head_size))


@functools.lru_cache(maxsize=256)
def _dims(*v) -> PaBiasedDims:
    _sizes(**{n: x for (n, t), x in zip(PaBiasedDims._fields_, v) if t is _i32})
    return PaBiasedDims(*v)


def _of_rows(t, name, n, dtype, index):
    """The address of an optional (n,) tensor."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.get_device() != index or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous ({n},) tensor on cuda:{index}")
    return t.data_ptr()


def biased_paged_attention(query: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                           cumulative_sequence_length: torch.Tensor, past_seqlens: torch.Tensor,
                           block_table: torch.Tensor, *, num_heads: int, kv_num_heads: int, scale: float = 0.0,
                           softcap: float = 0.0, slopes: Optional[torch.Tensor] = None, window: int = 0,
                           first_keys: Optional[torch.Tensor] = None, prefix_lens: Optional[torch.Tensor] = None,
                           max_query_len: int = 0, output: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                           error: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``paged_attention``'s read path with other scores and masks (pa_biased_paged_attention). The
    caches already hold this step's rows. A score ``scale * q.k`` becomes
    ``softcap * tanh(. / softcap)`` (``softcap`` > 0), then less ``slopes[h]`` (float32
    (num_heads,)) times the distance of the positions. A row at position p sees keys up to p, or
    up to ``prefix_lens`` (int32 (batch,)) where that is more (never past the sequence's end), from
    the latest of 0, ``p - window + 1`` (``window`` > 0) and ``first_keys`` (int32 (N,): the start
    of the row's document). A row that sees none gives zeros and an lse of -inf. The table's
    entries of pages that no row of a sequence sees may be anything. ``max_query_len`` (optional) is the host's bound on new
    rows per sequence. ``query`` may be a view of packed rows; ``lse`` (float32 (N, num_heads))
    receives the log-sum-exp; rows behind the last sequence are left as they were. ``workspace``
    (``biased_workspace_size(head_size)`` bytes): else the call allocates its own. A pipeline wait
    that runs out (DEVERR_TIMEOUT) is told by ``error`` only."""
    if output is None and workspace is None and stream is None:
        made = (step._fast or step._load_fast()).biased_paged_attention(
            query, key_cache, value_cache, cumulative_sequence_length, past_seqlens, block_table, num_heads, kv_num_heads,
            scale, softcap, slopes, window, first_keys, prefix_lens, max_query_len, lse, error)
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
    if output is None:
        output = _empty((N, num_heads * hs), dtype, query.device, stream)
    elif output.dtype is not dtype or output.get_device() != index or output.shape != (N, num_heads * hs) or \
            not output.is_contiguous():
        raise ValueError("output must be contiguous (rows, num_heads * head_size) of the query dtype")
    if lse is not None and (lse.dtype is not torch.float32 or lse.get_device() != index or lse.shape != (N, num_heads) or
                            not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 (rows, num_heads)")
    _sizes(window=window)
    for name, x in (("softcap", softcap), ("scale", scale)):  # (0 stands for no cap, and for the scale by the head size)
        if x != 0 and _f32(x).value == 0:
            raise ValueError(f"{name} is 0 in 32 bits")
    rules = PaScoreRules(softcap, window, _of_rows(slopes, "slopes", num_heads, torch.float32, index),
                         _of_rows(first_keys, "first_keys", N, torch.int32, index),
                         _of_rows(prefix_lens, "prefix_lens", B, torch.int32, index), 0)
    d = _dims(N, B, num_heads, kvh, hs, blocks, bs, columns, _T[dtype], max_query_len, stride, 0)
    lib = _library()
    ws = _workspace(workspace, lib.pa_biased_workspace_size(hs), index, query.device, stream)
    _call("pa_biased_paged_attention", index, stream, lib.pa_biased_paged_attention, query.data_ptr(),
          key_cache.data_ptr(), value_cache.data_ptr(), cumulative_sequence_length.data_ptr(), past_seqlens.data_ptr(),
          block_table.data_ptr(), scale, rules, output.data_ptr(), None if lse is None else lse.data_ptr(), d, err,
          ws.data_ptr(), ws.numel() * ws.element_size())
    return output
