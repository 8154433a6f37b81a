"""The operators around the attention call in the calls a serving loop makes of them: stages of the
dense call beside them, values that are not finite, host threads, sizes at the limits."""
import ctypes
import os
import subprocess
import threading

import numpy as np
import pytest
import torch

import varlen_paged_kv_gb300 as pa
from test_step_gpu import DT, Batch, f64, i32, run_tables, table_state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.fail("CUDA is required for the gpu tests")
    from varlen_paged_kv_gb300 import build
    build.build()


# ---- the cache write without the dense attention ---------------------------------------------


class Rows:
    """A batch with new rows still outside its caches."""

    def __init__(self, dtype, nh, kvh, hs, past, q, packed, bs=16):
        self.b = b = Batch(50, dtype, nh, kvh, hs, bs, past, q)
        b.key_cache.nan_to_num_(0)
        b.value_cache.nan_to_num_(0)
        g = torch.Generator().manual_seed(7)
        rows = torch.randn(b.N, (nh + 2 * kvh) * hs, generator=g).to(DT[dtype]).cuda()
        self.args = ((rows, None, None) if packed else
                     tuple(x.contiguous() for x in rows.split([nh * hs, kvh * hs, kvh * hs], 1)))
        self.new = [x.reshape(b.N, kvh, hs) for x in rows.split([nh * hs, kvh * hs, kvh * hs], 1)[1:]]
        dims = pa.make_dims(b.N, len(past), hs, b.blocks, bs, b.table.shape[1], DT[dtype], max_query_len=max(q))
        self.ws = torch.zeros(pa.workspace_size(dims, nh, kvh), dtype=torch.uint8, device="cuda")

    def call(self, stages, meta=None, bound=None):
        b = self.b
        pa.paged_attention(*self.args, b.key_cache, b.value_cache, *(meta or b.meta), num_heads=b.nh,
                           kv_num_heads=b.kvh, workspace=self.ws, max_query_len=bound or int(b.q.max()), stages=stages)

    def want(self, skip=()):
        """The caches with the new rows in their places, but those of the sequences in `skip`."""
        b, out = self.b, []
        for cache, rows in zip((b.key_cache, b.value_cache), self.new):
            c = cache.clone()
            for s in range(len(b.past)):
                for j in range(int(b.q[s]) if s not in skip else 0):
                    p = int(b.past[s]) + j
                    c[b.table[s, p // b.bs], p % b.bs] = rows[int(b.cum[s]) + j]
            out.append(c)
        return out

    def caches_are(self, want):
        return torch.equal(self.b.key_cache, want[0]) and torch.equal(self.b.value_cache, want[1])


STEPS = [("fp16", 8, 2, 128, [30, 50, 0, 15], [1, 1, 1, 1], False), ("bf16", 8, 2, 128, [30, 50, 0, 15], [1] * 4, True),
         ("fp16", 4, 4, 64, [3, 0, 100], [4, 1, 3], True), ("bf16", 16, 2, 256, [200, 31], [2, 2], False),
         ("fp16", 4, 4, 64, [20] * 300, [1] * 300, False)]  # (more sequences than plan themselves)


@pytest.mark.parametrize("dtype,nh,kvh,hs,past,q,packed", STEPS)
def test_the_cache_write_of_a_decode_step_stands_alone(dtype, nh, kvh, hs, past, q, packed):
    """A decode-only call that stops before its attention (another one reads the cache next) has written its rows."""
    for groups in ([pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE], [pa.STAGE_PLAN, pa.STAGE_CACHE_WRITE],
                   [pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE | pa.STAGE_PREFILL]):
        r = Rows(dtype, nh, kvh, hs, past, q, packed)
        want = r.want()
        for stages in groups:
            r.call(stages)
        assert pa.read_device_error(r.ws) == 0
        assert r.caches_are(want)
        r.call(pa.STAGE_DECODE)  # the rest of the same call
        assert pa.read_device_error(r.ws) == 0 and r.caches_are(want)


@pytest.mark.parametrize("packed", [False, True])
def test_a_refused_decode_step_writes_nothing_and_says_so(packed):
    past, q = [30, 50, 0, 15], [1, 1, 2, 1]
    for cum, lens, bound in (([0, 1, 2, 4, 6], past, 2), ([0, 1, 3, 2, 5], past, 2), (None, [30, -1, 0, 15], 2),
                             (None, [30, 5000, 0, 15], 2), (None, past, 1)):
        r = Rows("fp16", 8, 2, 128, past, q, packed)
        meta = (r.b.meta[0] if cum is None else i32(cum), i32(lens), r.b.meta[2])
        want = [r.b.key_cache.clone(), r.b.value_cache.clone()]
        r.call(pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE, meta, bound)
        assert pa.read_device_error(r.ws) == pa.DEVERR_BAD_BATCH and r.caches_are(want)
    # a page outside the pool: its row is dropped, the others are written
    r = Rows("fp16", 8, 2, 128, past, q, packed)
    table = r.b.table.copy()
    table[1, 50 // 16] = r.b.blocks
    want = r.want(skip=(1,))
    r.call(pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE, (*r.b.meta[:2], i32(table)))
    assert pa.read_device_error(r.ws) == pa.DEVERR_BAD_BLOCK and r.caches_are(want)


@pytest.mark.parametrize("kv_quant", ["int8", "int4"])
def test_a_refused_decode_step_on_integer_caches_says_so(kv_quant):
    b = Batch(51, "fp16", 8, 2, 128, 16, [30, 50], [1, 1])
    kc, vc = (torch.full((b.blocks, 16, 2, 128 if kv_quant == "int8" else 64), 77, dtype=torch.uint8, device="cuda")
              for _ in range(2))
    k = torch.randn(2, 256, device="cuda").half()
    s = torch.full((2, 128), 0.03, device="cuda")
    dims = pa.make_dims(2, 2, 128, b.blocks, 16, b.table.shape[1], torch.float16, max_query_len=1, kv_dtype=kv_quant)
    ws = torch.zeros(pa.workspace_size(dims, 8, 2), dtype=torch.uint8, device="cuda")
    pa.paged_attention(b.query.contiguous(), k, k, kc, vc, i32([0, 1, 3]), *b.meta[1:], num_heads=8, kv_num_heads=2,
                       workspace=ws, max_query_len=1, stages=pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE, kv_quant=kv_quant,
                       k_scale=s, v_scale=s)
    assert pa.read_device_error(ws) == pa.DEVERR_BAD_BATCH and (kc == 77).all() and (vc == 77).all()


def test_a_sparse_decode_step_with_derived_slots():
    """The decode call as the dense attention makes it, its attention replaced: what explicit slots give."""
    outs = []
    for derived in (True, False):
        r = Rows("bf16", 8, 2, 128, [100, 47, 64], [1, 1, 1], False)
        b = r.b
        if derived:
            r.call(pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE)
        else:
            slots = i32([b.table[s, b.past[s] // 16] * 16 + b.past[s] % 16 for s in range(3)])
            pa.paged_attention(*r.args, b.key_cache, b.value_cache, *b.meta, slots, num_heads=8, kv_num_heads=2,
                               stages=pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE)
        b.whole_bounds()
        sel = b.select(4)
        outs.append((b.bounds, sel, *b.attend(sel)))
    for x, y in zip(*outs):
        assert torch.equal(x, y)


# ---- values that are not finite --------------------------------------------------------------


def check_nan_rows(b, sel, R, bad, spoil, scale=0.0):
    """After spoil() the rows `bad` are NaN with an lse of NaN, and every other row is what it was within the bounds."""
    clean = b.attend(sel, R, scale)
    keep = [x.clone() for x in (b.rows, b.key_cache)]
    spoil()
    out, lse = b.attend(sel, R, scale)
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    b.rows.copy_(keep[0])
    b.key_cache.copy_(keep[1])
    out[bad], lse[bad] = clean[0][bad], clean[1][bad]
    b.check(out, lse, sel.cpu().numpy(), R, scale)
    assert int(b.error) == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("past,q,R", [([300, 2], [1, 1], 1),             # one list per CTA pair
                                      ([64 * 40, 700], [1, 3], 1),       # clusters
                                      ([64 * 40], [16], 16),             # clusters of tiles
                                      ([300, 0, 90], [20, 40, 1], 16)])
def test_a_query_of_nan_gives_nan(past, q, R, dtype):
    for scale in (0.0, -0.1):
        b = Batch(52, dtype, 8, 2, 128, 64, past, q, extra_rows=1)
        b.whole_bounds()
        sel = b.select(30, R)
        check_nan_rows(b, sel, R, [0], lambda: b.query[0].fill_(float("nan")), scale)
        last = int(b.cum[-1]) - 1

        def some_channels():
            for r in (0, last):
                b.query[r, ::16] = float("nan")

        check_nan_rows(b, sel, R, [0, last], some_channels, scale)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nh,kvh,hs,R", [(8, 2, 128, 1), (16, 2, 256, 1), (32, 2, 128, 4), (16, 2, 256, 4)])
def test_a_key_of_nan_gives_nan(nh, kvh, hs, R, dtype):
    """Where the key is the only one that a warp, a tile or a CTA of a cluster has, too."""
    nan = float("nan")
    for bs, past, n in ((16, 48, 1), (64, 64 * 20, 1), (64, 64 * 20 + 5, 130), (16, 16 * 33, 17)):
        b = Batch(53, dtype, nh, kvh, hs, bs, [past, 200], [1, 1])
        b.whole_bounds()
        sel = b.select(40, R)  # every page

        def spoil():
            for p in range(past - n + 1, past + 1):  # the last n keys
                b.key_cache[b.table[0, p // bs], p % bs] = nan

        check_nan_rows(b, sel, R, [0], spoil)
    # a key that only a block's last row sees
    if R == 4:
        b = Batch(54, dtype, nh, kvh, hs, 16, [47], [2])
        b.whole_bounds()
        sel = b.select(8, R)
        check_nan_rows(b, sel, R, [1], lambda: b.key_cache[b.table[0, 3], 0].fill_(nan))


# ---- sizes at the limits ---------------------------------------------------------------------


@pytest.mark.parametrize("free", [2, 0])
def test_block_tables_of_as_many_rows_as_there_can_be(free):
    """The last step of a loop over 2^31 - 2 rows ends past 2^31; also where the step is refused."""
    n = 2 ** 31 - 2
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    table = i32([[5, -1], [7, -1]])
    t = pa.build_block_tables(i32([15, 3]), i32([2, 1]), i32([1, 1]), table, i32([9, 4]), i32([1, free]), block_size=16,
                              num_tokens=n)
    torch.cuda.synchronize()
    assert int(t.error) == (0 if free else pa.DEVERR_NO_BLOCKS)
    rows = [[5 * 16 + 15, 4 * 16, 7 * 16 + 3], [15, 16, 3]] if free else [[], []]
    for got, want in zip((t.slot_mapping, t.positions), rows):
        assert got[: len(want)].tolist() == want
        for at in range(len(want), n, 1 << 28):
            assert int(got[at: at + (1 << 28)].max()) == -1 == int(got[at: at + (1 << 28)].min())
    assert t.cumulative_sequence_length.tolist() == ([0, 2, 3] if free else [0, 0, 0])
    assert t.blocks_held.tolist() == ([2, 1] if free else [1, 1]) and t.free_state.tolist() == ([0, 1] if free else [1, 0])
    assert table.tolist() == ([[5, 4], [7, -1]] if free else [[5, -1], [7, -1]])


# ---- host threads ----------------------------------------------------------------------------


def in_a_new_thread(f):
    """f() in a host thread of its own, where no other CUDA call has been made."""
    got = []

    def body():
        try:
            got.append(f())
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


@pytest.mark.parametrize("given", [False, True])  # outputs of the caller's, or of the call's
def test_first_calls_of_a_host_thread(given):
    """A thread's first call of the runtime gives it its context; no operator needs another call to have done so."""
    for R in (1, 16):
        b = Batch(61, "fp16", 8, 2, 128, 16, [300, 40], [20, 1])
        b.whole_bounds()
        sel = b.select(6, R)
        out, _ = b.attend(sel, R)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        kw = dict(num_heads=8, kv_num_heads=2, query_block=R)
        mine = dict(output=torch.empty_like(out), stream=side) if given else {}
        got = in_a_new_thread(lambda: pa.sparse_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, sel,
                                                                **kw, **mine))
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        mine = dict(selected=torch.empty_like(sel), stream=side) if given else {}
        got = in_a_new_thread(lambda: b.select(6, R, **mine))
        torch.cuda.synchronize()
        assert torch.equal(got, sel)
    t = table_state(np.random.default_rng(8), 9, 16, 8, 60, 20, 0.2)
    want, dev = run_tables(*t, 16, 200)
    again = in_a_new_thread(lambda: pa.build_block_tables(*dev, block_size=16, num_tokens=200,
                                                          out=want if given else None))
    torch.cuda.synchronize()
    assert torch.equal(again.slot_mapping, want.slot_mapping)
    q = b.query.contiguous()
    pos = i32(np.arange(len(q)))
    want = pa.qk_norm_rope(q, q[:, :256], pos, num_heads=8, kv_num_heads=2, rotary_dim=64)
    got = in_a_new_thread(lambda: pa.qk_norm_rope(q, q[:, :256], pos, num_heads=8, kv_num_heads=2, rotary_dim=64,
                                                  query_out=torch.empty_like(q) if given else None))
    kept = b.bounds.clone()
    in_a_new_thread(b.whole_bounds)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(b.bounds, kept)


def test_a_stage_of_the_dense_call_first_in_a_host_thread():
    r = Rows("fp16", 8, 2, 128, [30, 50], [1, 1], False)
    r.call(pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE)
    torch.cuda.synchronize()
    in_a_new_thread(lambda: r.call(pa.STAGE_DECODE))
    assert pa.read_device_error(r.ws) == 0


def table_calls(B, stream):
    """A function that calls build_block_tables for B requests, one that says whether its answer is right, and the
    arguments of the C entry point."""
    with torch.cuda.stream(stream):
        past, ones, held = (torch.full((B,), v, dtype=torch.int32, device="cuda") for v in (3, 1, 1))
        table = torch.arange(B, dtype=torch.int32, device="cuda").reshape(B, 1)
        ring, state = i32([0]), i32([0, 0])
        args = (past, ones, held, table, ring, state)
        out = pa.build_block_tables(*args, block_size=16, num_tokens=B)
        want = out.slot_mapping.clone()
    raw = (*args, B, B, 1, 16, 1, *out, stream.cuda_stream)
    return lambda: pa.build_block_tables(*args, block_size=16, num_tokens=B, out=out, stream=stream), \
        lambda: torch.equal(out.slot_mapping, want), raw


def select_calls(columns, top_k, stream, heads=8, kvh=2, hs=64):
    with torch.cuda.stream(stream):
        g = torch.Generator(device="cuda").manual_seed(columns)
        table = torch.randint(0, 64, (1, columns), generator=g, dtype=torch.int32, device="cuda")
        bounds = torch.randint(-127, 128, (64, kvh, 2, hs), generator=g, dtype=torch.int8, device="cuda")
        query = torch.randn(1, heads * hs, generator=g, device="cuda").half()
        scale, cum, past = torch.full((kvh, hs), 0.03, device="cuda"), i32([0, 1]), i32([columns * 16 - 1])
        kw = dict(num_heads=heads, kv_num_heads=kvh, block_size=16, top_k=top_k)
        sel = pa.select_pages(query, bounds, scale, cum, past, table, **kw)
        want = sel.clone()
    d = pa.PaSparseDims(1, 1, heads, kvh, hs, 64, 16, columns, 0, top_k, 1, 1, 1, 0, heads * hs)
    return lambda: pa.select_pages(query, bounds, scale, cum, past, table, selected=sel, stream=stream, **kw), \
        lambda: torch.equal(sel, want), (query, bounds, scale, cum, past, table, d, sel, 0, stream.cuda_stream)


def sparse_calls(top_k, R, stream):
    with torch.cuda.stream(stream):
        b = Batch(60, "fp16", 8, 2, 64, 16, [300], [R])
        sel = torch.full((b.N, 2, top_k), -1, dtype=torch.int32, device="cuda")
        sel[:, :, :19] = torch.arange(19, dtype=torch.int32, device="cuda")
        kw = dict(num_heads=8, kv_num_heads=2, query_block=R)
        args = (b.query, b.key_cache, b.value_cache, *b.meta, sel)
        out = pa.sparse_paged_attention(*args, **kw)
        want = out.clone()
    d = pa.PaSparseDims(b.N, 1, 8, 2, 64, b.blocks, 16, b.table.shape[1], 0, top_k, R, 0, 1, 0, 8 * 64)
    return lambda: pa.sparse_paged_attention(*args, output=out, stream=stream, **kw), \
        lambda: torch.equal(out, want), (*args, 0, out, 0, d, 0, stream.cuda_stream)


@pytest.fixture(scope="module")
def native(tmp_path_factory):
    """host_threads.cpp, compiled."""
    here = os.path.dirname(os.path.abspath(__file__))
    lib = str(tmp_path_factory.mktemp("native") / "host_threads.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I" + os.path.join(here, "..", "include"),
                    os.path.join(here, "host_threads.cpp"), "-o", lib], check=True)
    return ctypes.CDLL(lib)


@pytest.mark.parametrize("which,make,sizes", [
    (0, table_calls, [(8192,), (3000,)]), (1, select_calls, [(32000, 64), (5000, 32)]),
    (1, select_calls, [(4000, 64), (3400, 32)]), (2, sparse_calls, [(2048, 1), (32, 1)]),
    (2, sparse_calls, [(2048, 16), (32, 16)])])
def test_host_threads_with_calls_of_different_sizes(native, which, make, sizes):
    """A call's shared memory follows from its sizes; the limit that lets it launch is the function's, for all threads."""
    from varlen_paged_kv_gb300 import step
    calls = [make(*size, torch.cuda.Stream()) for size in sizes]
    torch.cuda.synchronize()
    lib = step._library()
    entry = (lib.pa_build_block_tables, lib.pa_select_pages, lib.pa_sparse_paged_attention)[which]
    raws = []
    for _, _, raw in calls:
        raws.append((ctypes.c_int64 * len(raw))(*[
            v.data_ptr() if torch.is_tensor(v) else ctypes.addressof(v) if isinstance(v, ctypes.Structure) else v
            for v in raw]))
    for _ in range(10):
        refused = native.two_threads(which, ctypes.cast(entry, ctypes.c_void_p), raws[0], raws[1], 500)
        torch.cuda.synchronize()
        assert refused == 0
    assert all(right() for _, right, _ in calls)


def test_a_graph_of_calls_of_different_sizes():
    """Both sizes of every kernel in one graph, and other sizes called between its capture and its replays."""
    side = torch.cuda.Stream()
    makes = [(table_calls, (8192,)), (table_calls, (3000,)), (select_calls, (32000, 64)), (select_calls, (5000, 32)),
             (select_calls, (40, 4)), (sparse_calls, (2048, 1)), (sparse_calls, (32, 1)), (sparse_calls, (2048, 16)),
             (sparse_calls, (32, 16))]
    calls = [make(*size, side) for make, size in makes]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for call, *_ in calls:
            call()
    for call, *_ in reversed(calls):
        call()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(right() for _, right, _ in calls)


def test_the_compiled_calls_let_other_threads_run(native):
    """An entry point that waits (as a launch does while the stream's queue is full) does not hold the interpreter."""
    from varlen_paged_kv_gb300 import step
    b = Batch(62, "fp16", 8, 2, 64, 16, [300], [2])
    b.whole_bounds()
    sel = b.select(5)
    fast, lib = step._load_fast(), step._library()
    real = [ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.pa_build_block_tables, lib.pa_qk_norm_rope, lib.pa_update_page_bounds, lib.pa_select_pages,
        lib.pa_sparse_paged_attention)]
    slow = ctypes.cast(native.slow_entry_point, ctypes.c_void_p).value
    one, q = i32([1]), b.query.contiguous()
    calls = [lambda: fast.build_block_tables(one, one, one, i32([[0]]), one, i32([0, 0]), 16, 1),
             lambda: fast.qk_norm_rope(q, q[:, :128], i32([0, 1]), 8, 2, None, None, 1e-6, 64, 1e4, False),
             lambda: fast.update_page_bounds(b.key_cache, b.bounds, b.scale, *b.meta, b.N, None),
             lambda: fast.select_pages(q, b.bounds, b.scale, *b.meta, 8, 2, 16, 5, 1, 1, 1, None),
             lambda: fast.sparse_paged_attention(q, b.key_cache, b.value_cache, *b.meta, sel, 8, 2, 0.0, 1, None, None)]
    try:
        for k, call in enumerate(calls):
            native.reset()
            fast.bind(*[slow if i == k else f for i, f in enumerate(real)])

            def other():
                while not native.has_entered():
                    pass
                native.release()

            t = threading.Thread(target=other)
            t.start()
            assert call() is not None, k  # (None: the call gave up before the other thread ran)
            t.join()
    finally:
        fast.bind(*real)
    torch.cuda.synchronize()


def test_sizes_past_32_bits_are_refused():
    """Not taken for their low 32 bits, which would be sizes that exist."""
    big = 1 << 32
    b = Batch(63, "fp16", 4, 2, 64, 16, [300], [2])
    b.whole_bounds()
    kw = dict(num_heads=4, kv_num_heads=2)
    sel = b.select(5)
    one = i32([1])
    for v in (big, -big):
        with pytest.raises(ValueError, match="block_size"):
            pa.build_block_tables(one, one, one, i32([[0]]), one, i32([0, 0]), block_size=16 + v, num_tokens=1)
        with pytest.raises(ValueError, match="rotary_dim"):
            pa.qk_norm_rope(b.query, b.query[:, :128], i32([0, 1]), rotary_dim=64 + v, **kw)
        with pytest.raises(ValueError, match="num_tokens"):
            pa.update_page_bounds(b.key_cache, b.bounds, b.scale, *b.meta, num_tokens=2 + v)
        with pytest.raises(ValueError, match="query_block"):
            pa.sparse_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, sel, query_block=1 + v, **kw)
        for name, x in (("block_size", 16), ("top_k", 5), ("query_block", 1), ("sink_pages", 1), ("local_pages", 1)):
            with pytest.raises(ValueError, match=name):
                pa.select_pages(b.query, b.bounds, b.scale, *b.meta, **kw, **(dict(block_size=16, top_k=5) | {name: x + v}))
    with pytest.raises(ValueError, match="num_tokens"):
        pa.build_block_tables(one, one, one, i32([[0]]), one, i32([0, 0]), block_size=16, num_tokens=big + 1)
    torch.cuda.synchronize()


# ---- a step of a fixed number of rows --------------------------------------------------------


@pytest.mark.parametrize("stages", [pa.STAGE_ALL, pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE])
def test_a_padded_step(stages):
    """16 rows for requests that fill 9: the dense call refuses the batch as it is; with a spare request for the other 7
    it writes and attends, and the others' rows are what they are without padding."""
    nh, kvh, hs, n = 8, 2, 64, 16
    g = torch.Generator().manual_seed(5)
    rows = torch.randn(n, (nh + 2 * kvh) * hs, generator=g).half().cuda()
    cache = [torch.randn(12, 16, kvh, hs, generator=g).half().cuda() for _ in range(2)]

    def step(past, q, held, n):
        B = len(past)
        kc, vc = (c.clone() for c in cache)
        table = i32([[3, 1, -1], [0, -1, -1], [-1, -1, -1]][:B])
        t = pa.build_block_tables(i32(past), i32(q), i32(held), table, i32([2, 4, 5, 6, 7, 8]), i32([0, 6]),
                                  block_size=16, num_tokens=n)
        assert int(t.error) == 0
        dims = pa.make_dims(n, B, hs, 12, 16, 3, torch.float16)
        ws = torch.zeros(pa.workspace_size(dims, nh, kvh), dtype=torch.uint8, device="cuda")
        out = torch.zeros(n, nh * hs, dtype=torch.float16, device="cuda")
        pa.paged_attention(rows[:n], None, None, kc, vc, t.cumulative_sequence_length, i32(past), table, t.slot_mapping,
                           num_heads=nh, kv_num_heads=kvh, output=out, workspace=ws, stages=stages)
        return kc, vc, out, pa.read_device_error(ws)

    kc, vc, out, error = step([30, 9], [4, 5], [2, 1], n)
    assert error == pa.DEVERR_BAD_BATCH and torch.equal(kc, cache[0]) and torch.equal(vc, cache[1]) and not out.any()
    want = step([30, 9], [4, 5], [2, 1], 9)
    got = step([30, 9, 0], [4, 5, 7], [2, 1, 0], n)
    assert want[3] == got[3] == 0
    mine = [3, 1, 0, 2]  # the two requests' pages; the spare one has taken 4
    for x, y in zip(want[:2], got[:2]):
        assert torch.equal(x[mine], y[mine]) and not torch.equal(x[4], y[4])
        assert not torch.equal(x, cache[0])
    if stages == pa.STAGE_ALL:
        assert torch.equal(got[2][:9], want[2][:9])


# ---- weights of very different sizes ---------------------------------------------------------


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits", [16.3, 24.4, 26.7, 30.2])
@pytest.mark.parametrize("nh,kvh,hs,R", [(8, 2, 64, 1), (8, 2, 64, 8), (16, 2, 256, 1), (16, 2, 256, 4)])
def test_small_weights_beside_a_large_one(nh, kvh, hs, R, bits, dtype):
    """One key with nearly all of the weight and a value of 0 beside thousands of 2^-bits each with values of 1 to 2:
    they make the output."""
    n, bs = 60 * 256, 256
    b = Batch(70, dtype, nh, kvh, hs, bs, [n - R], [R])
    b.whole_bounds()
    b.query.zero_()
    b.query[:, ::hs] = 16
    b.key_cache.zero_()
    g = torch.Generator().manual_seed(1)
    b.value_cache.copy_((1 + torch.rand(b.value_cache.shape, generator=g)).to(DT[dtype]))
    for at in (0, 100 * bs // 3, n - R):  # the large one: first, on the way, last for the block's first row
        page, off = b.table[0, at // bs], at % bs
        value = b.value_cache[page, off].clone()
        b.key_cache[page, off, :, 0], b.value_cache[page, off] = 16, 0
        scale = bits * np.log(2) / 256
        sel = i32(np.tile(np.arange(60), (R, kvh, 1)))
        out, lse = b.attend(sel, R, scale)
        k = np.arange(n)
        v = f64(b.value_cache[b.table[0, k // bs], torch.from_numpy(k % bs)])[:, None]          # (n, 1, kvh, hs)
        w = np.where(k[:, None] > n - R + np.arange(R), 0.0, 2.0 ** -bits)
        w[at] = 1.0
        total = w.sum(0)
        want = np.einsum("kr,kgc->rgc", w, v[:, 0]) / total[:, None, None]
        # the scores are exact but for the scale's rounding and the exponential's: 2^-22 of a score of `bits` each in
        # fp32, 2^-18 of a weight; a weight is rounded to fp16 (2^-11) or, below the subnormals' border, off by 2^-36
        # of the largest, or to two bf16 terms (2^-16); sums 2^-17; one rounding of the result
        half = torch.finfo(DT[dtype]).eps / 2
        weight = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -16
        small = 2 * n * 2.0 ** -36 if dtype == "fp16" else 0.0  # (values up to 2)
        bound = want * (half * (1 + 2.0 ** -7) + weight + 2.0 ** -18 + 2.0 ** -17) + small / total[:, None, None] + (
            2.0 ** -25 if dtype == "fp16" else 0.0)
        got = f64(out).reshape(R, kvh, nh // kvh, hs)
        assert (np.abs(got - want[:, :, None]) <= bound[:, :, None]).all(), (np.abs(got - want[:, :, None]) / bound[:, :, None]).max()
        z = np.log(total) + 256 * scale
        assert (np.abs(f64(lse) - z[:, None]) <= 2.0 ** -17 * (1 + np.abs(z[:, None]))).all()
        b.key_cache[page, off, :, 0], b.value_cache[page, off] = 0, value


def test_host_threads_each_with_its_own_steps():
    """Four threads, each with its stream, its batch and every operator: what each gives alone."""
    jobs = []
    for seed, (dtype, nh, kvh, hs, R, top_k) in enumerate([("fp16", 8, 2, 128, 1, 9), ("bf16", 16, 2, 256, 4, 30),
                                                           ("fp16", 8, 2, 64, 32, 200), ("bf16", 8, 8, 64, 1, 40)]):
        b = Batch(80 + seed, dtype, nh, kvh, hs, 16, [1500, 3000, 700], [1, 33, 2])
        b.whole_bounds()
        q, pos = b.query.contiguous(), i32(np.arange(b.N))
        tables = run_tables(*table_state(np.random.default_rng(seed), 30 * (seed + 1), 16, 20, 200, 40, 0.2), 16, 6000)[1]

        def job(b=b, q=q, pos=pos, tables=tables, R=R, top_k=top_k):
            sel = b.select(top_k, R)
            out = pa.sparse_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, sel, num_heads=b.nh,
                                            kv_num_heads=b.kvh, query_block=R)
            turned = pa.qk_norm_rope(q, q[:, : b.kvh * b.hs], pos, num_heads=b.nh, kv_num_heads=b.kvh, rotary_dim=b.hs)
            bounds = pa.update_page_bounds(b.key_cache, b.bounds.clone(), b.scale, *b.meta, num_tokens=b.N)
            return [sel, out, *turned, bounds, *pa.build_block_tables(*tables, block_size=16, num_tokens=6000)]

        jobs.append((job, job()))
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(jobs))

    def loop(job, want):
        start.wait()
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(100):
                    got = job()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(x, y) for x, y in zip(got, want)):
                        wrong.append("differs")
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=loop, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
