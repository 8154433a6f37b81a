"""The operators around the attention call: their refusals, on the host before any launch (so
none of this needs a GPU)."""
import ctypes

import pytest
import torch

import varlen_paged_kv_gb300 as pa
from varlen_paged_kv_gb300 import build

FAKE = 1 << 20  # aligned and never dereferenced: every case fails validation or has nothing to do


@pytest.fixture(scope="module")
def lib():
    build.build()
    from varlen_paged_kv_gb300 import step
    return step._library()


def tables(lib, B=4, N=8, cols=4, bs=16, cap=32, **ptr):
    names = ["past", "q", "held", "table", "ring", "state", "cum", "slots", "pos", "held_out", "state_out", "error"]
    a = {n: FAKE + 4096 * i for i, n in enumerate(names)} | ptr
    v = [a[n] for n in names]
    return lib.pa_build_block_tables(*v[:6], B, N, cols, bs, cap, *v[6:], None)


def test_block_tables_refusals(lib):
    assert tables(lib, B=-1) == 1 and tables(lib, N=-1) == 1 and tables(lib, bs=0) == 1 and tables(lib, cap=0) == 1
    assert tables(lib, cols=0) == 1
    assert tables(lib, B=8193) == 2                              # more requests than one call takes
    assert tables(lib, cols=1 << 28, bs=16) == 2                 # positions past 32 bits
    assert tables(lib, B=8192, cols=1 << 19) == 2                # a table past 32 bits of entries
    assert tables(lib, past=0) == 1 and tables(lib, error=0) == 1 and tables(lib, slots=FAKE + 2) == 1
    assert tables(lib, held_out=FAKE + 2 * 4096) == 1            # the old counts in place of the new ones
    assert tables(lib, state_out=FAKE + 5 * 4096) == 1


def rotate(lib, N=4, nh=8, kvh=2, hs=128, dt=0, d=64, theta=1e4, eps=1e-6, w=FAKE, q=FAKE, qs=1024, ks=256, qos=1024,
           kos=256, pos=FAKE, reserved=0):
    prep = pa.PaQkPrep(w, None, eps, theta, d, reserved)
    return lib.pa_qk_norm_rope(q, FAKE, pos, prep, 0, N, nh, kvh, hs, dt, qs, ks, FAKE, FAKE, qos, kos, None)


def test_qk_norm_rope_refusals(lib):
    assert rotate(lib, N=0) == 0                                 # nothing to do
    assert rotate(lib, N=-1) == 1 and rotate(lib, nh=0) == 1 and rotate(lib, reserved=1) == 1
    assert rotate(lib, hs=96) == 2 and rotate(lib, dt=2) == 2
    assert rotate(lib, d=24) == 2 and rotate(lib, d=144) == 2 and rotate(lib, d=-16) == 2
    assert rotate(lib, theta=0.0) == 1 and rotate(lib, eps=0.0) == 1
    assert rotate(lib, qs=1020) == 1 and rotate(lib, qs=1016) == 1 and rotate(lib, kos=248) == 1
    assert rotate(lib, q=FAKE + 8) == 1 and rotate(lib, pos=0) == 1 and rotate(lib, w=FAKE + 2) == 1


def dims(**kw):
    d = dict(num_tokens=8, batch_size=4, num_heads=8, kv_num_heads=2, head_size=128, num_blocks=64, block_size=64,
             max_blocks_per_sequence=16, dtype=0, top_k=4, query_block=1, sink_pages=1, local_pages=1, reserved=0,
             query_stride=1024)
    return pa.PaSparseDims(**(d | kw))


def call(lib, name, d, **ptr):
    a = dict(query=FAKE, key=FAKE, value=FAKE, bounds=FAKE, scale=FAKE, cum=FAKE, past=FAKE, table=FAKE, sel=FAKE,
             out=FAKE, lse=None, error=None) | ptr
    if name == "bounds":
        return lib.pa_update_page_bounds(a["key"], a["bounds"], a["scale"], a["cum"], a["past"], a["table"], d,
                                         a["error"], None)
    if name == "select":
        return lib.pa_select_pages(a["query"], a["bounds"], a["scale"], a["cum"], a["past"], a["table"], d, a["sel"],
                                   a["error"], None)
    return lib.pa_sparse_paged_attention(a["query"], a["key"], a["value"], a["cum"], a["past"], a["table"], a["sel"],
                                         0.0, a["out"], a["lse"], d, a["error"], None)


@pytest.mark.parametrize("name", ["bounds", "select", "sparse"])
def test_sparse_refusals(lib, name):
    assert call(lib, name, dims(num_tokens=0)) == 0
    assert call(lib, name, None) == 1
    for bad in (dict(num_tokens=-1), dict(batch_size=0), dict(num_heads=7), dict(kv_num_heads=0), dict(block_size=0),
                dict(num_blocks=0), dict(max_blocks_per_sequence=0), dict(reserved=1)):
        assert call(lib, name, dims(**bad)) == 1, bad
    for bad in (dict(head_size=96), dict(block_size=24), dict(dtype=2), dict(num_blocks=1 << 26),
                dict(max_blocks_per_sequence=1 << 26), dict(max_blocks_per_sequence=(1 << 25) - 1), dict(num_tokens=(1 << 31) - 5)):
        assert call(lib, name, dims(**bad)) == 2, bad
    for bad in (dict(cum=0), dict(past=FAKE + 2), dict(table=0), dict(error=FAKE + 1)):
        assert call(lib, name, dims(), **bad) == 1, bad
    if name == "bounds":
        assert call(lib, name, dims(), key=FAKE + 8) == 1 and call(lib, name, dims(), bounds=FAKE + 8) == 1
        return
    for bad in (dict(top_k=0), dict(query_block=0), dict(query_stride=1020), dict(query_stride=1016)):
        assert call(lib, name, dims(**bad)) == 1, bad
    for bad in (dict(top_k=2049), dict(query_block=257)):
        assert call(lib, name, dims(**bad)) == 2, bad
    assert call(lib, name, dims(), query=FAKE + 8) == 1 and call(lib, name, dims(), sel=0) == 1
    if name == "select":
        assert call(lib, name, dims(sink_pages=-1)) == 1 and call(lib, name, dims(local_pages=0)) == 1
        assert call(lib, name, dims(sink_pages=3, local_pages=2)) == 1           # more than top_k
        assert call(lib, name, dims(query_block=129, sink_pages=2, local_pages=1)) == 1   # the rows' own pages: 2 more
        assert call(lib, name, dims(max_blocks_per_sequence=32769)) == 2
    else:
        assert call(lib, name, dims(), out=0) == 1 and call(lib, name, dims(), lse=FAKE + 2) == 1


def test_python_refuses_host_tensors_and_wrong_types(lib):
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.build_block_tables(i, i, i, i.reshape(2, 1), i, i, block_size=16, num_tokens=1)
    h = torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        pa.qk_norm_rope(h, h, i, num_heads=1, kv_num_heads=1)
    c = torch.zeros(1, 16, 1, 64, dtype=torch.float16)
    b, s = torch.zeros(1, 1, 2, 64, dtype=torch.int8), torch.ones(1, 64)
    with pytest.raises(ValueError):
        pa.update_page_bounds(c, b, s, i, i[:1], i.reshape(1, 2), num_tokens=1)
    with pytest.raises(ValueError):
        pa.select_pages(h, b, s, i, i[:1], i.reshape(1, 2), num_heads=1, kv_num_heads=1, block_size=16, top_k=4)
    with pytest.raises(ValueError):
        pa.sparse_paged_attention(h, c, c, i, i[:1], i.reshape(1, 2), i.reshape(2, 1, 1), num_heads=1, kv_num_heads=1)


def test_the_struct_matches_the_header():
    assert ctypes.sizeof(pa.PaSparseDims) == 14 * 4 + 8
