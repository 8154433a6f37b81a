"""The page operators and the biased attention as a serving loop uses them: a prompt with a bidirectional prefix is
read once, forked into samples that share its pages, each sample decodes under a cap and a window, samples
replace one another and end, and the pool is compacted under them."""
import numpy as np
import pytest
import torch

import pool_reference as ref
import varlen_paged_kv_gb300 as pa
from test_step_gpu import _NoFast, f64, i32

pytestmark = pytest.mark.gpu
NH, KVH, HS, BS, COLS, BLOCKS = 8, 2, 128, 16, 24, 300


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.fail("CUDA is required for the gpu tests")
    from varlen_paged_kv_gb300 import build
    build.build()


class Loop:
    """The device's state of a batch of B requests, and each request's keys and values as the host knows them."""

    def __init__(self, B, seed):
        self.r = np.random.default_rng(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.kc, self.vc = (torch.zeros(BLOCKS, BS, KVH, HS, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.other = torch.zeros(BLOCKS, 4, dtype=torch.int32, device="cuda")  # (another layer's pages)
        self.past, self.held = i32(np.zeros(B)), i32(np.zeros(B))
        self.table, self.ring, self.state = i32(np.full((B, COLS), -1)), i32(np.arange(BLOCKS)), i32([0, BLOCKS])
        self.slopes = torch.from_numpy((2.0 ** -np.arange(1, NH + 1)).astype(np.float32)).cuda()
        self.text = [[np.zeros((0, KVH, HS))] * 2 for _ in range(B)]

    def step(self, q, **rules):
        """New rows for every request: their place, the cache write, the attention; checked against 64 bits."""
        q, n = np.asarray(q), int(np.sum(q))
        t = pa.build_block_tables(self.past, i32(q), self.held, self.table, self.ring, self.state, block_size=BS, num_tokens=n)
        assert int(t.error) == 0
        rows = torch.randn(n, (NH + 2 * KVH) * HS, generator=self.g).bfloat16().cuda()
        batch = (t.cumulative_sequence_length, self.past, self.table)
        pa.paged_attention(rows, None, None, self.kc, self.vc, *batch, t.slot_mapping, num_heads=NH, kv_num_heads=KVH,
                           stages=pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE)
        lse, error = torch.empty(n, NH, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        query = rows[:, : NH * HS]
        out = pa.biased_paged_attention(query, self.kc, self.vc, *batch, num_heads=NH, kv_num_heads=KVH, lse=lse, error=error,
                                        max_query_len=int(q.max()), slopes=self.slopes, **rules)
        assert int(error) == 0
        cum, past = t.cumulative_sequence_length.cpu().numpy(), self.past.cpu().numpy()
        k, v = (f64(rows)[:, (NH + i * KVH) * HS: (NH + (i + 1) * KVH) * HS].reshape(-1, KVH, HS) for i in range(2))
        kc, vc = np.full((BLOCKS, BS, KVH, HS), np.nan), np.full((BLOCKS, BS, KVH, HS), np.nan)
        table = np.full((len(q), COLS), -1)  # the host's own pages, one request after the other
        at = 0
        for b in range(len(q)):
            mine = slice(cum[b], cum[b + 1])
            self.text[b] = [np.concatenate([self.text[b][0], k[mine]]), np.concatenate([self.text[b][1], v[mine]])]
            for page in range(-(-len(self.text[b][0]) // BS)):
                table[b, page] = at
                for cache, text in ((kc, self.text[b][0]), (vc, self.text[b][1])):
                    part = text[page * BS: (page + 1) * BS]
                    cache[at, : len(part)] = part
                at += 1
        prefix = rules.get("prefix_lens")
        o, z, size, mag, far = ref.biased_attention(
            f64(query).reshape(n, NH, HS), kc, vc, cum, past, table, HS ** -0.5, rules.get("softcap", 0.0),
            self.slopes.cpu().numpy(), rules.get("window", 0), None, None if prefix is None else prefix.cpu().numpy())
        # (the bounds of test_biased_gpu, half a step of bf16 being 2^-8 of the value)
        cap = rules.get("softcap", 0.0)
        delta = mag * (HS + 8) * 2.0 ** -23 + cap * 2.0 ** -21 + far * 2.0 ** -22 + 2.0 ** -21 * (1 + np.abs(z) + cap)
        bound = 2.0 ** -8 * np.abs(o) * (1 + 2.0 ** -7) + size * (2.0 ** -16 + 2 * delta[..., None] + 2.0 ** -17)
        assert (np.abs(f64(out).reshape(o.shape) - o) <= bound).all()
        assert (np.abs(f64(lse) - z) <= delta + 2.0 ** -17).all()
        self.past, self.held, self.state = self.past + i32(q), t.blocks_held, t.free_state

    def fork(self, parents):
        f = pa.fork_block_tables(i32(parents), self.past, self.held, self.table, self.ring, self.state, block_size=BS,
                                 num_blocks=BLOCKS)
        assert int(f.error) == 0
        pa.copy_pages([self.kc, self.vc, self.other], f.copies)
        self.past, self.held, self.table, self.state = f.past_seqlens, f.blocks_held, f.block_table, f.free_state
        self.text = [list(self.text[p]) if p >= 0 else [np.zeros((0, KVH, HS))] * 2 for p in parents]

    def compact(self, moves):
        c = pa.compact_block_tables(self.held, self.table, self.ring, num_blocks=BLOCKS, max_moves=moves)
        assert int(c.error) == 0
        pa.copy_pages([self.kc, self.vc, self.other], c.copies)
        self.table, self.state = c.block_table, c.free_state
        return int(c.pages_end)

    def pages_in_use(self):
        held, table = self.held.cpu().numpy(), self.table.cpu().numpy()
        return {int(x) for b in range(len(held)) for x in table[b, : held[b]]}


@pytest.mark.parametrize("fast", [True, False])
def test_samples_of_shared_prompts(fast, monkeypatch):
    from varlen_paged_kv_gb300 import step
    if not fast:
        monkeypatch.setattr(step, "_fast", _NoFast())
    s = Loop(2, 3)
    s.step([75, 40], softcap=30.0, prefix_lens=i32([20, 300]))       # two prompts, the second read both ways
    assert len(s.pages_in_use()) == 5 + 3
    s.fork([0, 0, 0, 1, 1])                                          # five samples share their whole pages
    assert len(s.pages_in_use()) == 4 + 3 + 2 + 2
    for i in range(6):
        s.step([1, 1, 1, 1, 1], softcap=30.0, window=50)
    s.step([3, 1, 4, 2, 1], softcap=30.0, window=50)                 # drafts
    s.fork([2, 0, -1, 4, 2, 2])                                      # some replace others, some end
    s.step([1, 1, 9, 1, 1, 1], softcap=30.0)                         # (the empty row begins a new request)
    before = len(s.pages_in_use())
    assert s.compact(1000) == before and s.pages_in_use() == set(range(before))
    for i in range(4):
        s.step([1, 1, 1, 1, 1, 1], window=64)
    s.fork([5, 1, 0])
    s.compact(3)
    s.step([20, 1, 30], softcap=10.0)
    s.fork([-1, -1])
    assert not s.pages_in_use() and s.state.tolist()[1] == BLOCKS


def test_both_ways_into_the_library_agree(monkeypatch):
    """The compiled calls and the Python code behind them: the same results, types and shapes."""
    from varlen_paged_kv_gb300 import step
    from test_pool_gpu import pool_state
    from test_step_gpu import Batch

    def results():
        out = []
        for dtype, q in (("fp16", [1, 2]), ("bf16", [40, 7])):
            b = Batch(51, dtype, 8, 2, 128, 16, [300, 45], q, extra_rows=2, wide=256)
            lse = torch.zeros(b.N, 8, device="cuda")
            n = int(b.cum[-1])
            o = pa.biased_paged_attention(
                b.query, b.key_cache, b.value_cache, *b.meta, num_heads=8, kv_num_heads=2, scale=0.11, softcap=7.0, window=90,
                slopes=torch.arange(8, device="cuda") / 16.0, first_keys=i32(np.arange(b.N)), prefix_lens=i32([3, 50]),
                max_query_len=max(q), lse=lse, error=b.error)
            out += [o[:n], lse[:n], b.error]
        past, held, table, ring, state, blocks, pins = pool_state(np.random.default_rng(4), 30, 16, 20, 200, pinned=0.1)
        dev, pinned = [i32(v) for v in (past, held, table, ring, state)], torch.from_numpy(pins).cuda()
        f = pa.fork_block_tables(i32(np.arange(-1, 34) % 30), *dev, block_size=16, num_blocks=blocks, pinned=pinned)
        pages = torch.arange(blocks * 64, device="cuda", dtype=torch.int32).view(blocks, 64)
        pa.copy_pages((pages,), f.copies, error=f.error)
        c = pa.compact_block_tables(f.blocks_held, f.block_table, dev[3], num_blocks=blocks, max_moves=9, pinned=pinned)
        return out + list(f) + [pages] + list(c) + [dev[3]]

    fast = results()
    assert step._fast is not None
    monkeypatch.setattr(step, "_fast", _NoFast())
    slow = results()
    assert len(fast) == len(slow)
    for x, y in zip(fast, slow):
        assert x.dtype == y.dtype and x.shape == y.shape and x.is_contiguous() and torch.equal(x, y)


def test_refusals_say_what_was_wrong():
    from test_step_gpu import Batch
    b = Batch(52, "fp16", 4, 2, 64, 16, [100], [2])
    kw = dict(num_heads=4, kv_num_heads=2)
    call = lambda **k: pa.biased_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, **(kw | k))  # noqa: E731
    one = i32([1])
    for match, bad in (("slopes must be torch.float32", dict(slopes=torch.zeros(4, device="cuda", dtype=torch.float64))),
                       ("first_keys must be torch.int32", dict(first_keys=torch.zeros(2, device="cuda")))):
        with pytest.raises(TypeError, match=match):
            call(**bad)
    for match, bad in (("slopes must be", dict(slopes=torch.zeros(2, device="cuda"))), ("first_keys", dict(first_keys=one)),
                       ("prefix_lens", dict(prefix_lens=i32([1, 2]))), ("prefix_lens", dict(prefix_lens=torch.zeros(1).int())),
                       ("window must fit", dict(window=1 << 32)), ("max_query_len must fit", dict(max_query_len=1 << 40)),
                       ("lse", dict(lse=torch.zeros(2, 3).cuda())), ("output", dict(output=b.query[:1])),
                       ("cache shape", dict(kv_num_heads=1)), ("workspace", dict(workspace=torch.zeros(1 << 24, dtype=torch.uint8)))):
        with pytest.raises(ValueError, match=match):
            call(**bad)
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(window=-1), dict(scale=float("inf")), dict(max_query_len=-1)):
        with pytest.raises(pa.PagedAttentionError, match="INVALID_ARGUMENT"):
            call(**bad)
    with pytest.raises(pa.PagedAttentionError, match="WORKSPACE"):
        call(workspace=torch.zeros(100, dtype=torch.uint8, device="cuda"))
    t, tab = i32([20]), i32([[1, 2]])
    fork = lambda **k: pa.fork_block_tables(**(dict(parents=i32([0]), past_seqlens=t, blocks_held=i32([2]), block_table=tab,  # noqa: E731
                                                    free_blocks=i32([3]), free_state=i32([0, 1]), block_size=16,
                                                    num_blocks=8) | k))
    for match, bad in (("parents", dict(parents=i32([[0]]))), ("past_seqlens", dict(past_seqlens=i32([1, 2]))),
                       ("pinned", dict(pinned=torch.zeros(7, dtype=torch.bool, device="cuda"))),
                       ("num_blocks must fit", dict(num_blocks=1 << 33)), ("workspace", dict(workspace=torch.zeros(9999)))):
        with pytest.raises(ValueError, match=match):
            fork(**bad)
    with pytest.raises(TypeError, match="parents must be int32"):
        fork(parents=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError, match="pinned must be bool"):
        fork(pinned=torch.zeros(8, device="cuda"))
    good = fork()
    with pytest.raises(pa.PagedAttentionError, match="INVALID_ARGUMENT"):  # the old table is read while the new one is written
        fork(out=good._replace(block_table=tab))
    with pytest.raises(ValueError, match="out.copies"):
        fork(out=good._replace(copies=i32([[1, 2, 3]])))
    with pytest.raises(pa.PagedAttentionError, match="UNSUPPORTED"):
        fork(num_blocks=(1 << 20) + 1)
    with pytest.raises(ValueError, match="max_moves"):
        pa.compact_block_tables(i32([2]), tab, i32([3] * 8), num_blocks=8, max_moves=-1)
    with pytest.raises(ValueError, match="copies must be"):
        pa.copy_pages([b.key_cache], i32([1, 2]))
    with pytest.raises(ValueError, match="same pages"):
        pa.copy_pages([b.key_cache, b.key_cache[1:]], i32([[1, 2]]))
    with pytest.raises(ValueError, match="same pages"):
        pa.copy_pages([b.key_cache.transpose(0, 1)], i32([[1, 2]]))
    with pytest.raises(pa.PagedAttentionError, match="UNSUPPORTED"):  # pages of 10 bytes
        pa.copy_pages([torch.zeros(8, 10, dtype=torch.uint8, device="cuda")], i32([[1, 2]]))
    torch.cuda.synchronize()


def test_explicit_stream_argument():
    from test_step_gpu import Batch
    b = Batch(53, "fp16", 4, 2, 64, 16, [300, 60], [2, 50])
    kw = dict(num_heads=4, kv_num_heads=2, softcap=5.0)
    want = pa.biased_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, **kw)
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        # freed blocks of the current stream, still in use there, are not what the side stream writes to
        junk = torch.zeros(b.N, 256, dtype=torch.float16, device="cuda")
        for _ in range(20):
            busy = busy @ busy * 1e-3
        seen = junk.clone()
        del junk
        out = pa.biased_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, stream=side, **kw)
        side.synchronize()
        assert torch.equal(out, want) and (seen == 0).all()


def test_a_padded_step_is_captured_and_replayed():
    """A decode step with a fixed number of rows, some of them no one's, as a CUDA graph: replays on new lengths,
    masks and tables give what the calls give, and leave the rows behind alone."""
    from test_step_gpu import Batch
    b = Batch(54, "bf16", 8, 2, 128, 16, [300, 45, 90, 10], [1, 1, 1, 1], extra_rows=4)
    lse, out = torch.full((8, 8), 5.0, device="cuda"), torch.full((8, 1024), 5.0, dtype=torch.bfloat16, device="cuda")
    first, prefix = i32(np.zeros(8)), i32(np.zeros(4))
    ws = torch.empty(pa.biased_workspace_size(128), dtype=torch.uint8, device="cuda")

    def call(output, z):
        pa.biased_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, num_heads=8, kv_num_heads=2, softcap=9.0,
                                  first_keys=first, prefix_lens=prefix, output=output, lse=z, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out, lse)
    r = np.random.default_rng(1)
    for q in ([1, 1, 1, 1], [5, 1, 0, 2], [0, 0, 0, 0], [0, 8, 0, 0], [2, 2, 2, 2]):
        past = np.minimum([300, 45, 90, 10], r.integers(0, 301, 4))
        past = np.where(np.array(q) > 0, np.maximum(past + 1 - np.array(q), 0), past)
        b.meta[0].copy_(i32(np.concatenate([[0], np.cumsum(q)])))
        b.meta[1].copy_(i32(past))
        first.copy_(i32(r.integers(0, 40, 8)))
        prefix.copy_(i32(r.integers(0, 30, 4)))
        out.fill_(5)
        lse.fill_(5)
        o, z = out.clone(), lse.clone()
        graph.replay()
        torch.cuda.synchronize()
        call(o, z)
        n = sum(q)
        assert torch.equal(out, o) and torch.equal(lse, z)
        assert (out[n:] == 5).all() and (lse[n:] == 5).all()
        assert n == 0 or not (lse[:n] == 5).any()


@pytest.mark.parametrize("fast", [True, False])
def test_calls_with_nothing_to_do(fast, monkeypatch):
    """No rows, no new requests, no moves, no copies."""
    from varlen_paged_kv_gb300 import step
    if not fast:
        monkeypatch.setattr(step, "_fast", _NoFast())
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, ring, state = i(0, 1, 2, 3).view(2, 2), i(4, 5, 6, 7, 0, 0, 0, 0), i(0, 4)
    past, held = i(20, 32), i(2, 2)
    f = pa.fork_block_tables(i(), past, held, table, ring, state, block_size=16, num_blocks=8)
    assert f.block_table.shape == (0, 2) and f.copies.shape == (0, 2) and f.error.tolist() == [0]
    assert f.free_state.tolist() == [0, 8] and ring.tolist() == [4, 5, 6, 7, 0, 1, 2, 3]  # all pages back
    c = pa.compact_block_tables(held, table, ring, num_blocks=8, max_moves=0)
    assert c.copies.shape == (0, 2) and c.free_state.tolist() == [0, 4] and ring[:4].tolist() == [4, 5, 6, 7]
    assert c.pages_end.tolist() == [4] and torch.equal(c.block_table, table)
    cache = torch.randn(8, 16, 1, 64, device="cuda").half()
    was = cache.clone()
    pa.copy_pages([cache], torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    pa.copy_pages([cache], torch.full((3, 2), -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(cache, was)
    out = pa.biased_paged_attention(torch.empty(0, 128, device="cuda").half(), cache, cache, i(0, 0, 0), past, table, num_heads=2,
                                    kv_num_heads=1)
    assert out.shape == (0, 128)
    lse = torch.full((2, 2), 3.0, device="cuda")
    out = pa.biased_paged_attention(torch.zeros(2, 128, device="cuda").half(), cache, cache, i(0, 0, 0), past, table, num_heads=2,
                                    kv_num_heads=1, output=torch.full((2, 128), 4.0, device="cuda").half(), lse=lse)
    assert (out == 4).all() and (lse == 3).all()  # rows of no sequence


def test_host_threads_on_streams_of_their_own():
    """Eight threads call all four operators at once, each for a batch of its own: small kernels and large ones."""
    import threading
    wrong = []

    def work(k):
        try:
            r = np.random.default_rng(k)
            B, bs, blocks, cols = [6, 300][k % 2], 16, [200, 9000][k % 2], 24
            past = r.integers(1, bs * cols - 40, B)
            need = -(-past // bs)
            order = r.permutation(blocks)
            table, at = np.full((B, cols), -1), 0
            for b in range(B):
                table[b, :need[b]] = order[at: at + need[b]]
                at += need[b]
            free = order[at:]
            parents = r.integers(-1, B, B)
            q_len = [1, 3, 20, 1][k % 4]
            cum = np.arange(0, (4 + 1) * q_len, q_len)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                t = [i32(x) for x in (parents, past, need, table, np.concatenate([free, np.zeros(at, int)]), [0, len(free)])]
                key = torch.randn(blocks, bs, 2, 64, device="cuda").half()
                value = torch.randn(blocks, bs, 2, 64, device="cuda").half()
                query = torch.randn(4 * q_len, 512, device="cuda").half()
                first = None
                for _ in range(20):
                    ring, k2, v2 = t[4].clone(), key.clone(), value.clone()
                    f = pa.fork_block_tables(*t[:4], ring, t[5], block_size=bs, num_blocks=blocks)
                    pa.copy_pages([k2, v2], f.copies)
                    out = pa.biased_paged_attention(query, k2, v2, i32(cum), f.past_seqlens[:4] - f.past_seqlens[:4].clamp(max=q_len),
                                                    f.block_table[:4].contiguous(), num_heads=8, kv_num_heads=2, softcap=20.0,
                                                    window=100)
                    c = pa.compact_block_tables(f.blocks_held, f.block_table, ring, num_blocks=blocks, max_moves=64)
                    pa.copy_pages([k2, v2], c.copies)
                    got = [*f, *c, ring, k2, v2, out]
                    stream.synchronize()
                    first = first or [x.clone() for x in got]
                    assert int(f.error) == 0 and int(c.error) == 0
                    assert all(torch.equal(x, y) for x, y in zip(got, first))
        except Exception as e:  # noqa: BLE001 (an assertion of a thread is the test's)
            wrong.append((k, repr(e)))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(8)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not wrong, wrong
