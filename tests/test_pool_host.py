"""The operators on pages and the biased attention: their refusals, on the host before any launch."""
import ctypes

import pytest
import torch

import varlen_paged_kv_gb300 as pa
from varlen_paged_kv_gb300 import build

FAKE = 1 << 20  # aligned and never dereferenced: every case fails validation or has nothing to do
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    build.build()
    from varlen_paged_kv_gb300 import biased, pool
    pool._library()
    return biased._library()


def fork(lib, B=4, n=4, cols=4, bs=16, blocks=64, cap=64, ws_bytes=BIG, **ptr):
    names = ["parents", "past", "held", "table", "ring", "state", "pinned", "past_out", "held_out", "table_out",
             "copies", "state_out", "error", "ws"]
    a = {k: FAKE + 4096 * i for i, k in enumerate(names)} | ptr
    v = [a[k] for k in names]
    return lib.pa_fork_block_tables(*v[:7], B, n, cols, bs, blocks, cap, *v[7:], ws_bytes, None)


def test_fork_refusals(lib):
    for kw in (dict(B=-1), dict(n=-1), dict(cols=0), dict(bs=0), dict(blocks=0), dict(cap=0), dict(past=0), dict(parents=0),
               dict(ring=FAKE + 2), dict(copies=FAKE + 4), dict(ws=FAKE + 8), dict(ws=0), dict(error=0), dict(state_out=0)):
        assert fork(lib, **kw) == 1, kw
    same = {"past_out": 1, "held_out": 2, "table_out": 3, "state_out": 5}
    for name, i in same.items():  # rows are read while others are written
        assert fork(lib, **{name: FAKE + 4096 * i}) == 1
    for kw in (dict(B=8193), dict(n=8193), dict(blocks=(1 << 20) + 1), dict(cols=1 << 28), dict(n=8192, cols=1 << 19, bs=1),
               dict(cap=BIG + 1)):
        assert fork(lib, **kw) == 2, kw
    assert fork(lib, ws_bytes=lib.pa_pool_workspace_size(64) - 1) == 3


def compact(lib, B=4, cols=4, blocks=64, cap=64, moves=8, ws_bytes=BIG, **ptr):
    names = ["held", "table", "ring", "pinned", "table_out", "copies", "state_out", "end", "error", "ws"]
    a = {k: FAKE + 4096 * i for i, k in enumerate(names)} | ptr
    v = [a[k] for k in names]
    return lib.pa_compact_block_tables(*v[:4], B, cols, blocks, cap, moves, *v[4:], ws_bytes, None)


def test_compact_refusals(lib):
    for kw in (dict(B=-1), dict(cols=0), dict(blocks=0), dict(cap=0), dict(moves=-1), dict(held=0), dict(table_out=FAKE + 1),
               dict(copies=FAKE + 4), dict(end=0), dict(error=0), dict(ws=FAKE + 4)):
        assert compact(lib, **kw) == 1, kw
    for kw in (dict(B=8193), dict(blocks=(1 << 20) + 1), dict(moves=(1 << 20) + 1), dict(B=8192, cols=1 << 19)):
        assert compact(lib, **kw) == 2, kw
    assert compact(lib, ws_bytes=16) == 3
    assert lib.pa_pool_workspace_size(0) == 0 and lib.pa_pool_workspace_size((1 << 20) + 1) == 0


def copy(lib, tensors, n=3, blocks=10, copies=FAKE, error=FAKE):
    from varlen_paged_kv_gb300.pool import PaPageTensor
    t = (PaPageTensor * max(1, len(tensors)))(*[PaPageTensor(*x) for x in tensors])
    return lib.pa_copy_pages(t, len(tensors), blocks, copies, n, error, None)


def test_copy_refusals(lib):
    assert copy(lib, []) == 0 and copy(lib, [(FAKE, 64)], n=0) == 0  # nothing to do
    assert copy(lib, [(FAKE, 64)], n=-1) == 1 and copy(lib, [(FAKE, 64)], blocks=-1) == 1
    assert copy(lib, [(FAKE, 0)]) == 1 and copy(lib, [(FAKE + 8, 64)]) == 1 and copy(lib, [(0, 64)]) == 1
    assert copy(lib, [(FAKE, 64)], copies=FAKE + 4) == 1 and copy(lib, [(FAKE, 64)], error=FAKE + 1) == 1
    assert copy(lib, [(FAKE, 72)]) == 2 and copy(lib, [(FAKE, 1 << 31)]) == 2 and copy(lib, [(FAKE, 64)] * 257) == 2
    assert copy(lib, [(FAKE, 64)], n=(1 << 25) + 1) == 2


def attend(lib, ptr=None, ws_bytes=BIG, scale=0.0, rules=None, **kw):
    from varlen_paged_kv_gb300.biased import PaBiasedDims, PaScoreRules
    d = dict(num_tokens=8, batch_size=4, num_heads=8, kv_num_heads=2, head_size=128, num_blocks=64, block_size=64,
             max_blocks_per_sequence=16, dtype=0, max_query_len=0, query_stride=1024, reserved=0) | kw
    names = ["query", "k", "v", "cum", "past", "table", "out", "lse", "error", "ws"]
    a = {k: FAKE + 4096 * i for i, k in enumerate(names)} | (ptr or {})
    r = PaScoreRules(**(dict(softcap=0.0, window=0, slopes=None, first_keys=None, prefix_lens=None, reserved=0) |
                        (rules or {})))
    return lib.pa_biased_paged_attention(a["query"], a["k"], a["v"], a["cum"], a["past"], a["table"], scale, r, a["out"],
                                         a["lse"], PaBiasedDims(**d), a["error"], a["ws"], ws_bytes, None)


def test_biased_attention_refusals(lib):
    assert attend(lib, num_tokens=0) == 0  # nothing to do
    for kw in (dict(num_tokens=-1), dict(batch_size=0), dict(num_heads=7), dict(kv_num_heads=0), dict(block_size=0),
               dict(query_stride=1020), dict(query_stride=1016), dict(max_query_len=-1), dict(reserved=1), dict(num_blocks=0)):
        assert attend(lib, **kw) == 1, kw
    for kw in (dict(head_size=96), dict(dtype=2), dict(block_size=24), dict(num_blocks=1 << 26), dict(num_tokens=1 << 28),
               dict(num_heads=2050, kv_num_heads=1, head_size=64, query_stride=2050 * 64)):
        assert attend(lib, **kw) == 2, kw
    for name in ("query", "k", "v", "out", "ws"):
        assert attend(lib, ptr={name: FAKE + 8}) == 1 and attend(lib, ptr={name: 0}) == 1
    for name in ("cum", "past", "table"):
        assert attend(lib, ptr={name: 0}) == 1
    for name in ("lse", "error"):
        assert attend(lib, ptr={name: FAKE + 2}) == 1
    for rules in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(softcap=1e-35), dict(window=-1),
                  dict(slopes=FAKE + 2), dict(first_keys=FAKE + 1), dict(prefix_lens=FAKE + 2), dict(reserved=1)):
        assert attend(lib, rules=rules) == 1, rules
    assert attend(lib, scale=3e38) == 1 and attend(lib, scale=1e30, rules=dict(softcap=1e-10)) == 1
    assert attend(lib, scale=float("inf")) == 1 and attend(lib, scale=float("nan")) == 1
    assert attend(lib, ws_bytes=lib.pa_biased_workspace_size(128) - 1) == 3
    assert lib.pa_biased_workspace_size(96) == 0


def test_python_calls_refuse_host_tensors(lib):
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="block_table must be a CUDA tensor"):
        pa.fork_block_tables(i, i, i, t, i, i, block_size=16, num_blocks=8)
    with pytest.raises(ValueError, match="block_table must be a CUDA tensor"):
        pa.compact_block_tables(i, t, i, num_blocks=8, max_moves=1)
    with pytest.raises(ValueError, match="copies must be a CUDA tensor"):
        pa.copy_pages([torch.zeros(4, 16)], torch.zeros(1, 2, dtype=torch.int32))
    q = torch.zeros(2, 256, dtype=torch.float16)
    with pytest.raises(ValueError, match="query must be a CUDA tensor"):
        pa.biased_paged_attention(q, q, q, i, i, t, num_heads=2, kv_num_heads=2)
    assert pa.copy_pages([], None) is None
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_biased_attention_refuses_an_output_over_the_query(lib):
    out = FAKE + 4096 * 64
    rows, row = 4, 1024 * 2  # bytes of a row, 8 heads of 128

    def at(query, stride=1024):
        return attend(lib, ptr={"query": query, "out": out}, num_tokens=rows, query_stride=stride, num_heads=8,
                      kv_num_heads=2, head_size=128, ws_bytes=0)
    for query in (out, out + 16, out - 16, out + rows * row - 16, out - rows * row + 16):
        assert at(query) == 1
    assert at(out - 3 * 4 * row, stride=4096) == 1          # its last row is the output's first
    for query in (out + rows * row, out - rows * row):
        assert at(query) == 3                               # the workspace is what is refused


def test_biased_attention_refuses_more_blocks_than_a_grid_has(lib):
    assert attend(lib, batch_size=1 << 28, num_tokens=8) == 2
