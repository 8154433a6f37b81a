"""The operators on pages (forks, compactions, copies) against their plain statements
(pool_reference): whole numbers, and bytes, exactly."""
import numpy as np
import pytest
import torch

import pool_reference as ref
import varlen_paged_kv_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("CUDA is required for the gpu tests")
    from varlen_paged_kv_gb300 import build
    build.build()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def pool_state(r, B, bs, cols, longest, spare=40, share=0.5, pinned=0.0, extra=0.2, fit=False):
    """(past, held, table, ring, state, pages of the pool, pinned): requests that share some of their pages."""
    past = r.integers(0, longest + 1, B)
    held = np.minimum(-(-past // bs) + (r.random(B) < extra), cols)
    blocks = int(held.sum()) + spare
    order = r.permutation(blocks)
    table = np.full((B, cols), -1)
    at = 0
    for b in range(B):
        common = 0
        if b and r.random() < share:  # the whole pages of the row before
            common = min(past[b], past[b - 1]) // bs
            table[b, :common] = table[b - 1, :common]
        n = held[b] - common
        table[b, common: held[b]] = order[at: at + n]
        at += n
    free = order[at:]
    pins = r.random(blocks) < pinned
    free = free[~pins[free]]
    cap = blocks + (0 if fit else int(r.integers(0, 5)))
    ring, head = np.full(cap, -1), int(r.integers(0, cap))
    ring[(head + np.arange(len(free))) % cap] = free
    return past, held, table, ring, [head, len(free)], blocks, pins


def run_fork(parents, past, held, table, ring, state, bs, blocks, pinned=None, **kw):
    dev = [i32(v) for v in (parents, past, held, table, ring, state)]
    pins = None if pinned is None else torch.from_numpy(np.asarray(pinned)).cuda()
    return pa.fork_block_tables(*dev, block_size=bs, num_blocks=blocks, pinned=pins, **kw), dev


def check_fork(t, dev, want):
    for name, got in (("past", t.past_seqlens), ("held", t.blocks_held), ("table", t.block_table), ("copies", t.copies),
                      ("state", t.free_state), ("ring", dev[4])):
        assert np.array_equal(got.cpu().numpy(), np.asarray(want[name])), name
    assert int(t.error) == want["error"]


@pytest.mark.parametrize("B,n,bs,longest,pinned", [
    (1, 1, 16, 40, 0.0), (1, 9, 16, 37, 0.0), (5, 1, 48, 200, 0.3), (64, 64, 64, 4096, 0.0), (64, 100, 16, 500, 0.1),
    (300, 257, 256, 3000, 0.0), (700, 1100, 16, 100, 0.05), (40, 64, 16, 9000, 0.02), (8192, 8192, 16, 40, 0.01),
    (3, 0, 16, 100, 0.0), (7, 7, 16, 0, 0.5), (2500, 2600, 16, 300, 0.05), (120, 130, 16, 12000, 0.02), (5, 2049, 16, 90, 0.0)])
def test_fork(B, n, bs, longest, pinned):
    r = np.random.default_rng(B * 11 + n)
    past, held, table, ring, state, blocks, pins = pool_state(r, B, bs, -(-longest // bs) + 2, longest, spare=n + 40,
                                                             pinned=pinned)
    parents = np.where(r.random(n) < 0.2, -1, r.integers(0, B, n))
    want = ref.fork(parents, past, held, table, ring, state, bs, blocks, pins)
    assert want["error"] == 0 and (n < 100 or (want["copies"] >= 0).any())
    t, dev = run_fork(parents, past, held, table, ring, state, bs, blocks, pins)
    check_fork(t, dev, want)
    # the same call again gives the same, in outputs and a workspace of the caller's
    again = pa.ForkedTables(*[torch.full_like(x, 77) for x in t])
    ws = torch.full((pa.pool_workspace_size(blocks),), 255, dtype=torch.uint8, device="cuda")
    pa.fork_block_tables(*dev, block_size=bs, num_blocks=blocks, pinned=torch.from_numpy(pins).cuda(), out=again, workspace=ws)
    check_fork(again, dev, want)


def test_fork_no_old_rows():
    want = ref.fork([-1, -1], [], [], np.zeros((0, 4), int), np.arange(8), [3, 5], 16, 8)
    t, dev = run_fork([-1, -1], np.zeros(0), np.zeros(0), np.zeros((0, 4)), np.arange(8), [3, 5], 16, 8)
    check_fork(t, dev, want)


def test_fork_who_keeps_the_last_page():
    """Shared last pages, a last page that another row holds whole, a pinned one, lengths that were taken back."""
    bs, blocks = 16, 40
    table = np.full((5, 4), -1)
    table[0, :2] = 7, 9         # 20 tokens
    table[1, :3] = 7, 9, 11     # 40 tokens: holds row 0's last page whole
    table[2, :1] = 3            # 5 tokens
    table[3, :3] = 30, 31, 32   # taken back to 17 tokens: page 32 falls free
    table[4, :1] = 20           # 4 tokens, pinned
    past, held = [20, 40, 5, 17, 4], [2, 3, 1, 3, 1]
    pins = np.zeros(blocks, bool)
    pins[20] = True
    ring = np.arange(33, 40)
    roomy = np.full(30, -1)
    roomy[(26 + np.arange(7)) % 30] = ring
    for parents in ([0, 1, 2, 3, 4], [0, 0], [1, 0, 0, 1], [2, 2, 2], [4, 4], [3, 1, -1, 3], [-1] * 3):
        # (a ring without room behind its free pages refuses every fork that gives one back)
        for free, head in ((ring, 5), (roomy, 26)):
            want = ref.fork(parents, past, held, table, free, [head, 7], bs, blocks, pins)
            assert free is ring or want["error"] == 0
            t, dev = run_fork(parents, past, held, table, free, [head, 7], bs, blocks, pins)
            check_fork(t, dev, want)


@pytest.mark.parametrize("columns", [12, 200])  # one CTA's, and more
@pytest.mark.parametrize("what,code", [("parent", 1), ("parent low", 1), ("past", 1), ("held", 1), ("held low", 1),
                                       ("short", 1), ("page", 2), ("page low", 2), ("head", 1), ("count", 1), ("ring", 1),
                                       ("no pages", 16)])
def test_refused_forks_change_nothing(what, code, columns):
    r = np.random.default_rng(5)
    bs, B = 16, 600
    past, held, table, ring, state, blocks, _ = pool_state(r, B, bs, columns, 150, spare=700, fit=True)
    parents = r.integers(0, B, 700)
    past[599], held[599] = 20, 2
    table[599, :2] = 3, 4
    parents[3] = 599
    if what == "parent":
        parents[650] = B
    elif what == "parent low":
        parents[650] = -2
    elif what == "past":
        past[599] = -1
    elif what == "held":
        held[7] = columns + 1
    elif what == "held low":
        held[7] = -1
    elif what == "short":
        held[599] = 1
    elif what == "page":
        table[599, 1] = blocks
    elif what == "page low":
        table[599, 1] = -5
    elif what == "head":
        state[0] = len(ring)
    elif what == "count":
        state[1] = -1
    elif what == "ring":
        state[1] = len(ring)
        parents[:] = -1
    elif what == "no pages":
        state[1] = 3
    want = ref.fork(parents, past, held, table, ring, state, bs, blocks)
    assert want["error"] == code
    t, dev = run_fork(parents, past, held, table, ring, state, bs, blocks)
    check_fork(t, dev, want)


def run_compact(held, table, ring, blocks, max_moves, pinned=None, **kw):
    dev = [i32(v) for v in (held, table, ring)]
    pins = None if pinned is None else torch.from_numpy(np.asarray(pinned)).cuda()
    return pa.compact_block_tables(*dev, num_blocks=blocks, max_moves=max_moves, pinned=pins, **kw), dev


def check_compact(t, dev, want):
    for name, got in (("table", t.block_table), ("copies", t.copies), ("state", t.free_state), ("ring", dev[2])):
        assert np.array_equal(got.cpu().numpy(), np.asarray(want[name])), name
    assert int(t.pages_end) == want["end"] and int(t.error) == want["error"]


@pytest.mark.parametrize("B,bs,longest,spare,pinned", [
    (1, 16, 40, 3, 0.0), (1, 16, 0, 900, 0.0), (3, 48, 200, 40, 0.3), (64, 64, 4096, 900, 0.0), (64, 64, 4096, 2000, 0.1),
    (300, 16, 300, 4000, 0.02), (500, 16, 500, 9, 0.5), (8192, 16, 60, 30000, 0.01), (20, 16, 8000, 0, 0.0),
    (100, 16, 12000, 5000, 0.02), (2500, 48, 700, 0, 0.0), (3, 16, 100, 40000, 0.001)])
def test_compact(B, bs, longest, spare, pinned):
    r = np.random.default_rng(B * 13 + spare)
    _, held, table, ring, _, blocks, pins = pool_state(r, B, bs, -(-longest // bs) + 2, longest, spare=spare,
                                                      pinned=pinned)
    for limit in (0, 1, 33, blocks):
        want = ref.compact(held, table, ring, blocks, limit, pins)
        assert want["error"] == 0
        t, dev = run_compact(held, table, ring, blocks, limit, pins)
        check_compact(t, dev, want)
        # in place
        out = pa.CompactedTables(dev[1], *[torch.full_like(x, 77) for x in t[1:]])
        ws = torch.full((pa.pool_workspace_size(blocks),), 255, dtype=torch.uint8, device="cuda")
        pa.compact_block_tables(*dev, num_blocks=blocks, max_moves=limit, pinned=torch.from_numpy(pins).cuda(), out=out,
                                workspace=ws)
        check_compact(out, dev, want)


@pytest.mark.parametrize("blocks", [1, 31, 32, 33, 1023, 1024, 1025, 2048, 5000, 32768, 32769, 40001])
def test_compact_at_the_ends_of_words_and_chunks(blocks):
    """Any set of pages in use, one row each of one page, at pool sizes around a word of bits and a chunk of pages."""
    r = np.random.default_rng(blocks)
    for fill in (0.0, 0.03, 0.5, 0.97, 1.0):
        used = np.flatnonzero(r.random(blocks) < fill)
        used = r.permutation(used)[:8192]
        table = np.stack([used, np.full(len(used), -9)], 1)
        held, ring = np.ones(len(used), int), np.full(blocks, -3)
        pins = (r.random(blocks) < 0.1) if blocks > 40 else None
        want = ref.compact(held, table, ring, blocks, blocks, pins)
        t, dev = run_compact(held, table, ring, blocks, blocks, pins)
        check_compact(t, dev, want)


@pytest.mark.parametrize("columns", [12, 300])  # one CTA's, and more
@pytest.mark.parametrize("what,code", [("page", 2), ("page low", 2), ("held", 1), ("held low", 1), ("ring", 1)])
def test_refused_compactions_change_nothing(what, code, columns):
    r = np.random.default_rng(6)
    _, held, table, ring, _, blocks, _ = pool_state(r, 300, 16, columns, 150, spare=700)
    held[3] = 2
    table[3, :2] = 5, 6
    if what == "page":
        table[3, 1] = blocks
    elif what == "page low":
        table[3, 1] = -1
    elif what == "held":
        held[3] = columns + 1
    elif what == "held low":
        held[3] = -2
    elif what == "ring":
        ring = ring[:600]
    want = ref.compact(held, table, ring, blocks, 50)
    assert want["error"] == code
    t, dev = run_compact(held, table, ring, blocks, 50)
    check_compact(t, dev, want)


def test_the_largest_pool():
    """2^20 pages, the last of them in use and pinned among others."""
    blocks = 1 << 20
    table = np.array([[blocks - 1, 5, blocks - 2, 1 << 19], [0, 1, 7, -1]])
    pins = np.zeros(blocks, bool)
    pins[[blocks - 1, 3]] = True
    t, dev = run_compact([4, 3], table, np.full(blocks, -1), blocks, 100, pins)
    check_compact(t, dev, ref.compact([4, 3], table, np.full(blocks, -1), blocks, 100, pins))
    past = [50, 33]
    ring = np.full(blocks, -1)
    ring[:2] = 10, 11
    want = ref.fork([0, 0, 1], past, [4, 3], table, ring, [0, 2], 16, blocks, pins)
    t, dev = run_fork([0, 0, 1], past, [4, 3], table, ring, [0, 2], 16, blocks, pins)
    check_fork(t, dev, want)


# ---- copies ----------------------------------------------------------------------------------


def pages_of(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    return torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda", generator=g).view(dtype).view(shape)


@pytest.mark.parametrize("blocks,entries,shapes", [
    (1, 1, [((16,), torch.uint8)]), (40, 17, [((16, 2, 64), torch.float16), ((2, 2, 64), torch.int8), ((4,), torch.float32)]),
    (300, 1100, [((64, 8, 128), torch.bfloat16)] * 3), (70, 30, [((8208,), torch.uint8), ((16384,), torch.uint8)]),
    (9, 4, [(((1 << 20) + 48,), torch.uint8)]), (64, 32, [((16, 1, 64), torch.bfloat16)] * 256)])
def test_copy_pages(blocks, entries, shapes):
    r = np.random.default_rng(blocks + entries)
    tensors = [pages_of((blocks, *s), d, 5 + i) for i, (s, d) in enumerate(shapes)]
    before = [t.clone() for t in tensors]
    pages = r.permutation(blocks)
    pairs = pages[: blocks // 2 * 2].reshape(-1, 2)
    copies = np.full((entries, 2), -1)
    at = np.sort(r.permutation(entries)[: min(len(pairs), entries // 2 + 1)])
    copies[at] = pairs[: len(at)]
    error = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.copy_pages(tensors, i32(copies), error=error)
    for t, old in zip(tensors, before):
        want = old.clone()
        for a, b in copies[at]:
            want[b] = old[a]
        assert torch.equal(t.view(torch.uint8), want.view(torch.uint8))
    assert int(error) == 0


def test_copy_pages_one_source_to_many_and_to_itself():
    t = pages_of((10, 16, 2, 64), torch.float16, 1)
    old = t.clone()
    pa.copy_pages([t], i32([[3, 4], [3, 5], [3, 9], [7, 7]]))
    for i in (4, 5, 9):
        assert torch.equal(t[i].view(torch.int16), old[3].view(torch.int16))
    keep = [0, 1, 2, 3, 6, 7, 8]
    assert torch.equal(t[keep].view(torch.int16), old[keep].view(torch.int16))


def test_copy_pages_skips_and_reports_pages_outside_the_pool():
    t = pages_of((10, 16, 2, 64), torch.float16, 2)
    old, error = t.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.copy_pages([t], i32([[3, 10], [-1, 4], [5, -1], [-7, 2], [1 << 30, 0], [1, 2]]), error=error)
    assert int(error) == pa.DEVERR_BAD_BLOCK
    assert torch.equal(t[2].view(torch.int16), old[1].view(torch.int16))
    keep = [0, 1] + list(range(3, 10))
    assert torch.equal(t[keep].view(torch.int16), old[keep].view(torch.int16))
    pa.copy_pages([t], i32([[3, 10]]))  # nobody asks


def test_copy_pages_past_32_bits_of_bytes():
    t = torch.zeros(70, 1 << 25, dtype=torch.int16, device="cuda")  # 4.7 GB
    t[69] = 3
    t[1] = 5
    pa.copy_pages([t], i32([[69, 2], [1, 68]]))
    assert int(t[2].min()) == 3 and int(t[68].min()) == 5 and int(t[67].max()) == 0 and int(t[3].max()) == 0


# ---- together --------------------------------------------------------------------------------


def test_many_forks_and_compactions_keep_every_requests_tokens():
    """Requests fork, end, grow through build_block_tables and are compacted, on the device's state alone: every
    request reads its own tokens back, no page that it writes is shared, and no page is lost or free twice."""
    r = np.random.default_rng(1)
    B, bs, cols, blocks = 24, 16, 16, 330
    cache, other = torch.zeros(blocks, bs, dtype=torch.int32, device="cuda"), torch.zeros(blocks, 4, dtype=torch.int32, device="cuda")
    past, held, table = i32(np.zeros(B)), i32(np.zeros(B)), i32(np.full((B, cols), -1))
    ring, state = i32(np.arange(blocks)), i32([0, blocks])
    text = [[] for _ in range(B)]  # what each request has written
    token = 1
    for step in range(60):
        lens = [len(x) for x in text]
        q = np.where(np.array(lens) > 150, 0, r.integers(0, 9, B))
        n = int(q.sum())
        t = pa.build_block_tables(past, i32(q), held, table, ring, state, block_size=bs, num_tokens=n)
        assert int(t.error) == 0
        new = torch.arange(token, token + n, dtype=torch.int32, device="cuda")
        cache.view(-1)[t.slot_mapping.long()] = new
        at = 0
        for b in range(B):
            text[b] += list(range(token + at, token + at + q[b]))
            at += q[b]
        token += n
        past, held, state = past + i32(q), t.blocks_held, t.free_state
        # a third of the rows are replaced by others, some end
        parents = np.where(r.random(B) < 0.3, r.integers(0, B, B), np.arange(B))
        parents = np.where(r.random(B) < 0.08, -1, parents)
        f = pa.fork_block_tables(i32(parents), past, held, table, ring, state, block_size=bs, num_blocks=blocks)
        assert int(f.error) == 0
        pa.copy_pages([cache, other], f.copies)
        text = [list(text[p]) if p >= 0 else [] for p in parents]
        past, held, table, state = f.past_seqlens, f.blocks_held, f.block_table, f.free_state
        if step % 3 == 2:
            c = pa.compact_block_tables(held, table, ring, num_blocks=blocks, max_moves=int(r.integers(0, 60)))
            assert int(c.error) == 0
            pa.copy_pages([cache, other], c.copies)
            table, state = c.block_table, c.free_state
        h, tab, (head, count) = held.cpu().numpy(), table.cpu().numpy(), state.tolist()
        used = [set(tab[b, : h[b]]) for b in range(B)]
        free = ring.cpu().numpy()[(head + np.arange(count)) % blocks]
        assert len(set(free)) == count and not set(free) & set().union(*used)
        assert count + len(set().union(*used)) == blocks
        writes = [tab[b, len(text[b]) // bs] for b in range(B) if len(text[b]) % bs]
        assert len(set(writes)) == len(writes)
        for b in range(B):
            if len(text[b]) % bs:
                assert all(tab[b, len(text[b]) // bs] not in used[o] for o in range(B) if o != b)
            got = cache[table[b, : h[b]].long()].flatten()[: len(text[b])].tolist()
            assert got == text[b]


def test_forks_captured_and_replayed_and_on_another_stream():
    r = np.random.default_rng(8)
    past, held, table, ring, state, blocks, pins = pool_state(r, 50, 16, 20, 300, spare=120, pinned=0.05)
    dev = [i32(v) for v in (r.integers(-1, 50, 60), past, held, table, ring, state)]
    pinned = torch.from_numpy(pins).cuda()
    cache = pages_of((blocks, 16, 2, 64), torch.float16, 3)
    start = cache.clone()

    def step():
        f = pa.fork_block_tables(*dev, block_size=16, num_blocks=blocks, pinned=pinned)
        pa.copy_pages([cache], f.copies)
        c = pa.compact_block_tables(f.blocks_held, f.block_table, dev[4], num_blocks=blocks, max_moves=30, pinned=pinned)
        pa.copy_pages([cache], c.copies)
        return f, c

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        f, c = step()
    for seed in range(4):
        parents = np.random.default_rng(seed).integers(-1, 50, 60)
        dev[0].copy_(i32(parents))
        dev[4].copy_(i32(ring))
        cache.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        want = ref.fork(parents, past, held, table, ring, state, 16, blocks, pins)
        assert want["error"] == 0
        check_fork(f, [None] * 4 + [i32(want["ring"])], want)
        again = ref.compact(want["held"], want["table"], want["ring"], blocks, 30, pins)
        check_compact(c, [None, None, dev[4]], again)
        moved = start.clone()
        for pairs in (want["copies"], again["copies"]):
            for a, b in pairs[pairs[:, 0] >= 0]:
                moved[b] = moved[a].clone()
        assert torch.equal(cache.view(torch.int16), moved.view(torch.int16))
    # an explicit stream
    dev[4].copy_(i32(ring))
    torch.cuda.synchronize()
    f = pa.fork_block_tables(*dev, block_size=16, num_blocks=blocks, pinned=pinned, stream=side)
    pa.copy_pages([cache], f.copies, stream=side)
    side.synchronize()
    check_fork(f, [None] * 4 + [dev[4]], want)
