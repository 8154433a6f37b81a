"""The operators around the attention call against their plain statements (step_reference):
whole numbers exactly, the rest within bounds derived from the roundings."""
import numpy as np
import pytest
import torch

import step_reference as ref
import varlen_paged_kv_gb300 as pa

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("CUDA is required for the gpu tests")
    from varlen_paged_kv_gb300 import build
    build.build()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


# ---- block tables ----------------------------------------------------------------------------


def table_state(r, B, bs, cols, longest, chunk, finished, spare=64, extra=0.1):
    past = r.integers(0, longest + 1, B)
    q = np.where(r.random(B) < 0.5, 1, r.integers(0, chunk + 1, B))
    q = np.where(r.random(B) < finished, -1, q)
    held = np.minimum(-(-past // bs) + (r.random(B) < extra), cols)
    need = np.where(q > 0, -(-(past + np.maximum(q, 0)) // bs), 0)
    free = int(np.maximum(need - held, 0).sum()) + spare
    blocks = int(held.sum()) + free
    order = r.permutation(blocks)
    table = np.full((B, cols), -1)
    at = 0
    for b in range(B):
        table[b, : held[b]] = order[at: at + held[b]]
        at += held[b]
    cap = blocks + int(r.integers(0, 5))
    ring, head = np.full(cap, -1), int(r.integers(0, cap))
    ring[(head + np.arange(free)) % cap] = order[at:]
    return past, q, held, table, ring, [head, free]


def run_tables(past, q, held, table, ring, state, bs, N, out=None):
    dev = [i32(v) for v in (past, q, held, table, ring, state)]
    t = pa.build_block_tables(*dev, block_size=bs, num_tokens=N, out=out)
    return t, dev


def check_tables(t, dev, want):
    for name, got in (("cum", t.cumulative_sequence_length), ("slots", t.slot_mapping), ("positions", t.positions),
                      ("held", t.blocks_held), ("state", t.free_state), ("table", dev[3]), ("ring", dev[4])):
        assert np.array_equal(got.cpu().numpy(), np.asarray(want[name])), name
    assert int(t.error) == want["error"]


@pytest.mark.parametrize("B,bs,longest,chunk,finished,pad", [
    (1, 16, 0, 1, 0.0, 0), (1, 256, 4096, 700, 0.0, 5), (3, 16, 40, 33, 0.3, 1), (64, 256, 4096, 1, 0.0, 0),
    (511, 48, 900, 40, 0.1, 64), (512, 16, 300, 1, 0.5, 0), (513, 16, 300, 5, 0.0, 7), (1200, 64, 4096, 300, 0.05, 129),
    (8192, 16, 64, 4, 0.1, 3), (5, 16, 100, 0, 1.0, 9)])
def test_block_tables(B, bs, longest, chunk, finished, pad):
    r = np.random.default_rng(B * 7 + bs)
    a = table_state(r, B, bs, -(-(longest + max(chunk, 1)) // bs) + 1, longest, chunk, finished)
    N = int(np.maximum(a[1], 0).sum()) + pad
    t, dev = run_tables(*a, bs, N)
    want = ref.block_tables(*a, bs, N)
    assert want["error"] == 0
    check_tables(t, dev, want)
    # the same call again gives the same
    again = pa.build_block_tables(*dev, block_size=bs, num_tokens=N)
    check_tables(again, dev, want)


def test_block_tables_no_requests_and_no_rows():
    a = (np.zeros(0), np.zeros(0), np.zeros(0), np.zeros((0, 4)), np.arange(8), [3, 5])
    t, dev = run_tables(*a, 16, 6)
    check_tables(t, dev, ref.block_tables(a[0], a[1], a[2], np.zeros((0, 4), int), np.arange(8), [3, 5], 16, 6))
    a = table_state(np.random.default_rng(5), 4, 16, 8, 60, 0, 0.5)
    a = a[:1] + (np.minimum(a[1], 0),) + a[2:]
    t, dev = run_tables(*a, 16, 0)
    check_tables(t, dev, ref.block_tables(*a, 16, 0))


@pytest.mark.parametrize("what,code", [("no blocks", 16), ("rows", 1), ("past", 1), ("q", 1), ("columns", 1), ("held", 1),
                                       ("head", 1), ("count", 1), ("ring", 1), ("huge", 1)])
def test_block_tables_refused_steps_change_nothing(what, code):
    r = np.random.default_rng(11)
    past, q, held, table, ring, state = table_state(r, 700, 16, 12, 100, 40, 0.1, spare=0)
    q[5], past[5], held[5] = 17, 0, 0
    N = int(np.maximum(q, 0).sum())
    if what == "no blocks":
        state[1] -= 1
        held[5] = 0
    elif what == "rows":
        N -= 1
    elif what == "past":
        past[699] = -1
    elif what == "q":
        q[699] = -2
    elif what == "columns":
        past[3], q[3] = 12 * 16, 1
    elif what == "held":
        held[8] = 13
    elif what == "head":
        state[0] = len(ring)
    elif what == "count":
        state[1] = -1
    elif what == "ring":
        state[1] = len(ring)
        q[1], held[1] = -1, 1
    elif what == "huge":  # the sum of the lengths passes 32 bits
        q[:] = 2 ** 31 - 1
        past[:] = 0
    a = (past, q, held, table, ring, state)
    t, dev = run_tables(*a, 16, N)
    want = ref.block_tables(*a, 16, N)
    assert want["error"] == code
    check_tables(t, dev, want)


def test_block_tables_invalid_page_gives_no_slot():
    table = np.array([[3, -1, 5], [1 << 30, 2, 0]])
    t, _ = run_tables([15, 3], [2, 1], [2, 1], table, np.arange(4), [0, 0], 16, 3)
    assert t.slot_mapping.tolist() == [3 * 16 + 15, -1, -1] and t.positions.tolist() == [15, 16, 3]


def test_block_tables_over_many_steps():
    """Requests come, grow and leave on the device's state alone: no page has two owners."""
    r = np.random.default_rng(3)
    B, bs, cols, blocks = 40, 16, 16, 200
    past, held, table = np.zeros(B, int), i32(np.zeros(B)), i32(np.full((B, cols), -1))
    ring, state = i32(r.permutation(blocks)), i32([0, blocks])
    for step in range(30):
        q = np.where(r.random(B) < 0.2, r.integers(1, 40, B), 1)
        q = np.where((r.random(B) < 0.1) | (past + q > cols * bs), -1, q)
        t = pa.build_block_tables(i32(past), i32(q), held, table, ring, state, block_size=bs, num_tokens=2000)
        if int(t.error):
            q = np.where(np.arange(B) % 3 == 0, -1, 0)  # make room
            t = pa.build_block_tables(i32(past), i32(q), held, table, ring, state, block_size=bs, num_tokens=2000)
            assert int(t.error) == 0
        past = np.where(q < 0, 0, past + np.maximum(q, 0))
        held, state = t.blocks_held.clone(), t.free_state.clone()
        h, tab, (head, count) = held.cpu().numpy(), table.cpu().numpy(), state.tolist()
        free = ring.cpu().numpy()[(head + np.arange(count)) % blocks]
        owned = np.concatenate([tab[b, : h[b]] for b in range(B)])
        assert sorted(np.concatenate([owned, free])) == list(range(blocks))


# ---- norm and rotation -----------------------------------------------------------------------


def rotate_bound(y, size, dtype):
    """One rounding to T, and fp32 arithmetic: at most 20 roundings of 2^-24 on the values that enter (the sum of
    squares 13 / 2, sqrt, quotient and two products 4, sine and cosine 4, two products and a sum 3), below 2^-19."""
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0  # half of fp16's least step
    return torch.finfo(DT[dtype]).eps / 2 * np.abs(y) * (1 + 2.0 ** -8) + 2.0 ** -19 * size + tiny


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nh,kvh,hs,d", [(32, 8, 128, 128), (16, 2, 256, 64), (3, 1, 64, 16), (16, 16, 64, 64),
                                         (5, 5, 256, 256), (7, 1, 128, 48), (4, 2, 128, 0), (1, 1, 64, 32)])
def test_qk_norm_rope(nh, kvh, hs, d, dtype, interleaved):
    for n, packed, norm in ((1, False, True), (5, True, False), (67, True, True), (400, False, True)):
        g = torch.Generator().manual_seed(nh * hs + n)
        rows = torch.randn(n, (nh + 2 * kvh) * hs, generator=g).to(DT[dtype]).cuda()
        q, k = rows[:, : nh * hs], rows[:, nh * hs: (nh + kvh) * hs]
        if not packed:
            q, k = q.contiguous(), k.contiguous()
        pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32).cuda()
        pos[0] = 0
        wq = (1 + torch.randn(hs, generator=g) / 4).to(DT[dtype]).cuda() if norm else None
        wk = (1 + torch.randn(hs, generator=g) / 4).to(DT[dtype]).cuda() if norm and n != 67 else None
        qo, ko = pa.qk_norm_rope(q, k, pos, num_heads=nh, kv_num_heads=kvh, q_norm_weight=wq, k_norm_weight=wk,
                                 eps=1e-5, rotary_dim=d, theta=1e6, interleaved=interleaved)
        for x, w, heads, got in ((q, wq, nh, qo), (k, wk, kvh, ko)):
            y, size = ref.norm_rope(f64(x).reshape(n, heads, hs), None if w is None else f64(w),
                                    float(np.float32(1e-5)), pos.cpu().numpy(), d, 1e6, interleaved)
            assert (np.abs(f64(got).reshape(y.shape) - y) <= rotate_bound(y, size, dtype)).all()
        # in place on the rows as they lie gives the same bits and leaves V
        keep = rows.clone()
        a, b = pa.qk_norm_rope(q, k, pos, num_heads=nh, kv_num_heads=kvh, q_norm_weight=wq, k_norm_weight=wk, eps=1e-5,
                               rotary_dim=d, theta=1e6, interleaved=interleaved, query_out=q, key_out=k)
        assert a is q and b is k and torch.equal(q, qo) and torch.equal(k, ko)
        assert torch.equal(rows[:, (nh + kvh) * hs:], keep[:, (nh + kvh) * hs:])


def test_qk_norm_rope_at_far_positions():
    """Angles of many thousand turns: the 32-bit product with the position defines them, its sine is exact to 2^-21."""
    pos = np.array([0, 1, 105615, 105616, 131071, (1 << 24) - 1, (1 << 24) + 1, 1 << 30, (1 << 31) - 1])
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn(len(pos), 64 * h, generator=g).half().cuda() for h in (3, 1))
    got = pa.qk_norm_rope(q, k, i32(pos), num_heads=3, kv_num_heads=1, rotary_dim=64, theta=1e4)
    for x, h, y in ((q, 3, got[0]), (k, 1, got[1])):
        want, size = ref.norm_rope(f64(x).reshape(-1, h, 64), None, 1e-6, pos, 64, 1e4, False)
        assert (np.abs(f64(y).reshape(want.shape) - want) <= rotate_bound(want, size, "fp16")).all()


def test_qk_norm_rope_leaves_rows_of_no_sequence():
    q = torch.randn(6, 256).half().cuda()
    k = torch.randn(6, 64).half().cuda()
    pos = i32([3, -1, 0, 7, -1, -1])
    qo, ko = torch.full_like(q, 9), torch.full_like(k, 9)
    pa.qk_norm_rope(q, k, pos, num_heads=4, kv_num_heads=1, rotary_dim=64, query_out=qo, key_out=ko)
    gone = (pos < 0).cpu()
    assert (qo[gone] == 9).all() and (ko[gone] == 9).all() and not (qo[~gone] == 9).all(1).any()
    assert torch.equal(qo[2], q[2]) and torch.equal(ko[2], k[2])  # position 0 turns nothing


def test_qk_norm_rope_matches_the_attention_calls_preparation():
    """paged_attention's own preparation writes the same prepared keys to its cache."""
    nh, kvh, hs, n = 8, 2, 128, 33
    g = torch.Generator().manual_seed(1)
    q = torch.randn(n, nh * hs, generator=g).half().cuda()
    k, v = (torch.randn(n, kvh * hs, generator=g).half().cuda() for _ in range(2))
    w = (1 + torch.randn(hs, generator=g) / 4).half().cuda()
    caches = [torch.zeros(4, 16, kvh, hs, dtype=torch.float16, device="cuda") for _ in range(2)]
    table = i32([[2, 0, 3, 1]])
    pa.paged_attention(q, k, v, *caches, i32([0, n]), i32([10]), table, num_heads=nh, kv_num_heads=kvh,
                       qk_prep=dict(q_norm_weight=w, k_norm_weight=w, eps=1e-6, rotary_dim=64, theta=1e4))
    _, ko = pa.qk_norm_rope(q, k, i32(10 + np.arange(n)), num_heads=nh, kv_num_heads=kvh, q_norm_weight=w,
                            k_norm_weight=w, eps=1e-6, rotary_dim=64, theta=1e4)
    p = 10 + np.arange(n)
    got = caches[0][table[0].cpu().numpy()[p // 16], p % 16].reshape(n, kvh * hs)
    # each is within half a step of the exact value, so they are at most one step apart
    step = 2.0 ** (torch.floor(torch.log2(ko.double().abs().clamp(min=2.0 ** -14))) - 10)
    assert ((got.double() - ko.double()).abs() <= step * 1.001).all()


# ---- paged batches ---------------------------------------------------------------------------


class Batch:
    def __init__(self, seed, dtype, nh, kvh, hs, bs, past, q, extra_rows=0, extra_pages=3, wide=0, spread=1.0):
        r = np.random.default_rng(seed)
        self.nh, self.kvh, self.hs, self.bs, self.dtype = nh, kvh, hs, bs, dtype
        self.past, self.q = np.asarray(past), np.asarray(q)
        self.cum = np.concatenate([[0], np.cumsum(self.q)])
        self.N = int(self.cum[-1]) + extra_rows
        pages = -(-(self.past + self.q) // bs)
        self.blocks = int(pages.sum()) + extra_pages
        order = r.permutation(self.blocks)
        self.table = np.full((len(past), max(1, int(pages.max()) + 1)), -1)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at: at + n]
            at += n
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: (torch.randn(*s, generator=g) * spread).to(DT[dtype]).cuda()  # noqa: E731
        self.rows = rand(self.N, nh * hs + wide)
        self.query = self.rows[:, : nh * hs]
        self.key_cache, self.value_cache = (rand(self.blocks, bs, kvh, hs) for _ in range(2))
        # rows that no sequence reaches hold NaN: none of it may show
        for b in range(len(past)):
            end = int(self.past[b] + self.q[b])
            if end % bs:
                self.key_cache[self.table[b, end // bs], end % bs:] = float("nan")
                self.value_cache[self.table[b, end // bs], end % bs:] = float("nan")
        for p in order[at:]:
            self.key_cache[p] = self.value_cache[p] = float("nan")
        self.scale = torch.from_numpy(r.uniform(0.02, 0.05, (kvh, hs)).astype(np.float32)).cuda()
        self.bounds = torch.zeros(self.blocks, kvh, 2, hs, dtype=torch.int8, device="cuda")
        self.meta = (i32(self.cum), i32(self.past), i32(self.table))
        self.error = torch.zeros(1, dtype=torch.int32, device="cuda")

    def whole_bounds(self):
        """The bounds of everything cached: one call from an empty past."""
        total = self.past + self.q
        cum = np.concatenate([[0], np.cumsum(total)])
        pa.update_page_bounds(self.key_cache, self.bounds, self.scale, i32(cum), i32(0 * self.past), self.meta[2],
                              num_tokens=int(cum[-1]), error=self.error)
        return cum

    def select(self, top_k, R=1, **kw):
        return pa.select_pages(self.query, self.bounds, self.scale, *self.meta, num_heads=self.nh,
                               kv_num_heads=self.kvh, block_size=self.bs, top_k=top_k, query_block=R,
                               error=self.error, **kw)

    def want_selected(self, top_k, R=1, sink_pages=1, local_pages=1, fill=-7):
        return ref.select_pages(self.query.float().cpu().numpy().reshape(self.N, self.nh, self.hs),
                                self.bounds.cpu().numpy(), self.scale.cpu().numpy(), self.cum, self.past, self.table,
                                self.kvh, self.bs, top_k, R, sink_pages, local_pages, fill)

    def attend(self, selected, R=1, scale=0.0, **kw):
        lse = torch.full((self.N, self.nh), 5.0, device="cuda")
        out = torch.full((self.N, self.nh * self.hs), 5.0, dtype=DT[self.dtype], device="cuda")
        pa.sparse_paged_attention(self.query, self.key_cache, self.value_cache, *self.meta, selected,
                                  num_heads=self.nh, kv_num_heads=self.kvh, scale=scale, query_block=R, output=out,
                                  lse=lse, error=self.error, **kw)
        return out, lse

    def check(self, out, lse, selected, R=1, scale=0.0):
        sc = scale or self.hs ** -0.5
        o, z, size, mag = ref.sparse_attention(f64(self.query).reshape(self.N, self.nh, self.hs), f64(self.key_cache),
                                               f64(self.value_cache), self.cum, self.past, self.table,
                                               np.asarray(selected), sc, R)
        n = int(self.cum[-1])
        got, gz = f64(out).reshape(o.shape), f64(lse)
        assert (got[n:] == 5).all() and (gz[n:] == 5).all()  # rows behind the last sequence
        o, z, size, mag, got, gz = o[:n], z[:n], size[:n], mag[:n], got[:n], gz[:n]
        # scores: hs products summed in fp32 (at most one unit of 2^-23 of the sum of magnitudes a step), the scale
        # and the exponential 2^-21; each weight enters P V rounded to fp16 (half a step, 2^-11) or as two bf16 terms
        # (2^-16); sums over the keys and the merge of partial results 2^-18; then one rounding to T
        delta = mag * (self.hs + 8) * 2.0 ** -23 + 2.0 ** -21 * (1 + np.where(np.isfinite(z), np.abs(z), 0))
        weight = 2.0 ** -11 if self.dtype == "fp16" else 2.0 ** -16
        eps = torch.finfo(DT[self.dtype]).eps / 2
        tiny = 2.0 ** -25 if self.dtype == "fp16" else 0.0
        bound = eps * np.abs(o) * (1 + 2.0 ** -7) + size * (weight + 2 * delta[..., None] + 2.0 ** -17) + tiny
        assert (np.abs(got - o) <= bound).all(), (np.abs(got - o) / bound).max()
        some = np.isfinite(z)
        assert np.array_equal(np.isneginf(gz), ~some)
        assert (np.abs(gz[some] - z[some]) <= (delta + 2.0 ** -17)[some]).all()


SHAPES = [(8, 2, 128, 64), (4, 4, 64, 16), (16, 2, 256, 32), (6, 2, 128, 48), (32, 2, 64, 128), (20, 1, 128, 16)]


# ---- bounds ----------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nh,kvh,hs,bs", SHAPES)
def test_page_bounds(nh, kvh, hs, bs, dtype):
    past = [0, 5, bs, 3 * bs - 1, 2 * bs + 7, 0, 200]
    q = [1, 2 * bs + 3, 1, 2, 0, 3 * bs, 5]
    b = Batch(1, dtype, nh, kvh, hs, bs, past, q, extra_rows=2)
    r = np.random.default_rng(2)
    b.bounds.copy_(torch.from_numpy(np.sort(r.integers(-128, 128, b.bounds.shape), 2).astype(np.int8)))
    start, keys = b.bounds.cpu().numpy(), b.key_cache.float().cpu().numpy()
    got = pa.update_page_bounds(b.key_cache, b.bounds, b.scale, *b.meta, num_tokens=b.N, error=b.error)
    want = ref.page_bounds(keys, start, b.scale.cpu().numpy(), b.cum, b.past, b.table)
    assert got is b.bounds and np.array_equal(got.cpu().numpy(), want) and int(b.error) == 0
    pa.update_page_bounds(b.key_cache, b.bounds, b.scale, *b.meta, num_tokens=b.N)
    assert np.array_equal(b.bounds.cpu().numpy(), want)  # again: the same
    # from an empty past: the bounds of the whole cache, as built up step by step
    cum = b.whole_bounds()
    assert np.array_equal(b.bounds.cpu().numpy(), ref.page_bounds(keys, want, b.scale.cpu().numpy(), cum,
                                                                  0 * b.past, b.table))


def test_page_bounds_special_keys():
    b = Batch(3, "fp16", 2, 1, 64, 16, [0], [20])
    k = b.key_cache[b.table[0, 0]]
    k[3, 0, 5], k[4, 0, 6], k[5, 0, 7] = float("nan"), float("inf"), -float("inf")
    k[:, 0, 9], k[:, 0, 10] = -0.0, float("nan")
    keys = b.key_cache.float().cpu().numpy()
    pa.update_page_bounds(b.key_cache, b.bounds, b.scale, *b.meta, num_tokens=b.N)
    want = ref.page_bounds(keys, np.zeros(b.bounds.shape), b.scale.cpu().numpy(), b.cum, b.past, b.table)
    assert np.array_equal(b.bounds.cpu().numpy(), want)
    assert want[b.table[0, 0], 0, :, 10].tolist() == [127, -127]  # no key counts


def test_bad_batches_are_skipped_and_reported():
    b = Batch(4, "fp16", 4, 2, 64, 16, [30, 10, 40], [3, 2, 4])
    b.whole_bounds()
    sel = b.select(4).cpu().numpy()
    out, lse = b.attend(i32(sel))
    for cum, past, table, bit in (([0, 3, 5, 11], b.past, b.table, 1), (b.cum, [30, 10, -1], b.table, 1),
                                  (b.cum, [30, 10, 4000], b.table, 1),
                                  (b.cum, b.past, np.where(np.arange(3)[:, None] == 2, 1 << 20, b.table), 2)):
        meta = (i32(cum), i32(past), i32(table))
        kept = b.bounds.clone()
        e = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(3)]
        pa.update_page_bounds(b.key_cache, kept, b.scale, *meta, num_tokens=b.N, error=e[0])
        s = pa.select_pages(b.query, b.bounds, b.scale, *meta, num_heads=4, kv_num_heads=2, block_size=16, top_k=3,
                            error=e[1])
        o, z = torch.zeros_like(out), torch.zeros_like(lse)
        pa.sparse_paged_attention(b.query, b.key_cache, b.value_cache, *meta, i32(sel), num_heads=4, kv_num_heads=2,
                                  output=o, lse=z, error=e[2])
        # (the third sequence's three pages are all selected, so none is scored and looked up)
        assert [int(x) & bit for x in e] == [bit, 0 if bit == 2 else bit, bit]
        assert torch.equal(kept, b.bounds)
        assert torch.equal(o[:5], out[:5]) and torch.equal(z[:5], lse[:5])  # the other sequences
        assert (s[:5] >= -1).all()
        if bit == 2:  # no page is in the pool: nothing to attend
            assert (o[5:] == 0).all() and torch.isneginf(z[5:]).all()


def test_scored_pages_outside_the_pool_are_reported():
    b = Batch(14, "fp16", 4, 2, 64, 16, [16 * 20], [1])
    b.whole_bounds()
    b.table[0, 7] = b.blocks
    meta = (b.meta[0], b.meta[1], i32(b.table))
    s = pa.select_pages(b.query, b.bounds, b.scale, *meta, num_heads=4, kv_num_heads=2, block_size=16, top_k=4,
                        error=b.error)
    assert int(b.error) == pa.DEVERR_BAD_BLOCK
    s = s.cpu().numpy()
    assert (s[..., 0] == 0).all() and (s[..., -1] == 20).all() and (np.diff(s, axis=2) > 0).all()


# ---- selection -------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nh,kvh,hs,bs", SHAPES)
@pytest.mark.parametrize("R", [1, 4, 33])
def test_select_pages(nh, kvh, hs, bs, R, dtype):
    past = [0, 7 * bs + 3, 40 * bs - 1, 11 * bs, 3, 23 * bs + 5]
    q = [1, 70, 1, 0, 40, 9]
    b = Batch(5, dtype, nh, kvh, hs, bs, past, q, extra_rows=3, wide=16)
    b.whole_bounds()
    for top_k, sink, local in ((2 + -(-(R - 1) // bs), 1, 1), (9, 0, 2), (64, 3, 4)):
        out = torch.full((b.N, kvh, top_k), -7, dtype=torch.int32, device="cuda")
        got = b.select(top_k, R, sink_pages=sink, local_pages=local, selected=out)
        assert got is out
        assert np.array_equal(out.cpu().numpy(), b.want_selected(top_k, R, sink, local))
    assert int(b.error) == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_select_of_many_blocks(dtype):
    """Thousands of selections, so that products that round to a half on the way to their code occur by the score."""
    b = Batch(15, dtype, 16, 4, 64, 16, [16 * 300 + 5, 16 * 150, 16 * 600], [1500, 1600, 1501])
    b.whole_bounds()
    assert np.array_equal(b.select(24, 4).cpu().numpy(), b.want_selected(24, 4))


def test_select_ties_go_to_the_lowest_page():
    b = Batch(6, "fp16", 4, 2, 128, 16, [16 * 900 + 3, 16 * 3], [1, 5])
    r = np.random.default_rng(7)
    b.bounds.copy_(torch.from_numpy(r.integers(0, 2, b.bounds.shape[:1] + (1, 1, 1)).astype(np.int8) * 50))  # two scores
    for top_k in (2, 5, 400, 600, 902):
        assert np.array_equal(b.select(top_k).cpu().numpy(), b.want_selected(top_k))
    b.bounds.zero_()
    assert np.array_equal(b.select(6).cpu().numpy(), b.want_selected(6))
    b.bounds[:, :, 0], b.bounds[:, :, 1] = -128, 127  # the largest scores there are
    b.query.fill_(1)
    assert np.array_equal(b.select(6).cpu().numpy(), b.want_selected(6))


@pytest.mark.parametrize("fill", [0.0, 1e-8, float("nan"), float("inf"), 6e4])
def test_select_special_queries(fill):
    b = Batch(8, "fp16", 8, 2, 64, 16, [16 * 50 + 1, 30], [3, 6])
    b.whole_bounds()
    b.query[1] = fill
    b.query[2, ::3] = fill
    b.query[5, :70] = fill
    for R in (1, 2):
        assert np.array_equal(b.select(7, R).cpu().numpy(), b.want_selected(7, R))


@pytest.mark.parametrize("pages,top_k", [(8192, 128), (8190, 2048), (32767, 2), (2048, 1000)])
def test_select_long_histories(pages, top_k):
    """Long histories in few distinct pages of the pool (the bounds of a page serve many times)."""
    r = np.random.default_rng(pages)
    past = [16 * (pages - 1) + 5, 16 * (pages // 3) + 15]
    table = r.integers(0, 500, (2, pages))
    bounds = np.sort(r.integers(-127, 128, (500, 2, 2, 64)), 2).astype(np.int8)
    q = torch.randn(3, 8 * 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    scale = np.full((2, 64), 0.03, np.float32)
    got = pa.select_pages(q, torch.from_numpy(bounds).cuda(), torch.from_numpy(scale).cuda(), i32([0, 1, 3]), i32(past),
                          i32(table), num_heads=8, kv_num_heads=2, block_size=16, top_k=top_k)
    want = ref.select_pages(q.float().cpu().numpy().reshape(3, 8, 64), bounds, scale, [0, 1, 3], past, table, 2, 16,
                            top_k, 1, 1, 1)
    assert np.array_equal(got.cpu().numpy(), want)


# ---- attention over the selection ------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nh,kvh,hs,bs", SHAPES)
@pytest.mark.parametrize("R", [1, 4, 33])
def test_sparse_attention(nh, kvh, hs, bs, R, dtype):
    past = [0, 7 * bs + 3, 20 * bs - 1, 11 * bs, 3, 13 * bs + 5]
    q = [1, 70, 1, 0, 40, 9]
    b = Batch(9, dtype, nh, kvh, hs, bs, past, q, extra_rows=3, wide=16)
    b.whole_bounds()
    for top_k, scale in ((2 + -(-(R - 1) // bs), 0.0), (9, -0.2), (37, 0.3)):
        sel = b.select(top_k, R)
        out, lse = b.attend(sel, R, scale)
        b.check(out, lse, sel.cpu().numpy(), R, scale)
        again, _ = b.attend(sel, R, scale)
        assert torch.equal(out, again)
    assert int(b.error) == 0


@pytest.mark.parametrize("nh,kvh,hs,bs,past,q,top_k,R", [
    (8, 2, 128, 16, [16 * 2300 + 3], [1], 2048, 1),       # the longest list, few rows: clusters
    (16, 2, 256, 16, [16 * 2300 + 3], [5], 2048, 5),      # and 256-wide heads on the tile kernel
    (16, 2, 256, 16, [16 * 700 + 3], [1], 600, 1),
    (4, 4, 64, 16, [16 * 500], [40], 300, 20),
    (2, 2, 64, 512, [5000, 0], [1, 700], 6, 128),         # long pages, blocks longer than the sequence
    (4, 1, 128, 16, [5], [1], 15, 200),                   # a block of 800 rows, a batch of one
    (160, 1, 64, 32, [300, 7], [3, 1], 5, 1),             # more heads per group than a tile has rows
    (160, 1, 64, 32, [300, 7], [3, 9], 5, 6),
    (12, 2, 128, 80, [1000, 401], [7, 30], 8, 7)])        # pages of 80: segments of 16 keys
def test_sparse_attention_at_the_edges(nh, kvh, hs, bs, past, q, top_k, R):
    for dtype in ("fp16", "bf16"):
        b = Batch(31, dtype, nh, kvh, hs, bs, past, q, extra_rows=1)
        b.whole_bounds()
        sel = b.select(top_k, R)
        assert np.array_equal(sel.cpu().numpy()[: int(b.cum[-1])], b.want_selected(top_k, R)[: int(b.cum[-1])])
        out, lse = b.attend(sel, R)
        b.check(out, lse, sel.cpu().numpy(), R)
        assert int(b.error) == 0


@pytest.mark.parametrize("nh,kvh,hs,R", [(8, 2, 128, 1), (8, 2, 128, 32), (16, 2, 256, 16), (8, 8, 64, 64)])
def test_sparse_attention_again_and_again(nh, kvh, hs, R):
    """The same call many times over, the GPU busy with others between: the same bits every time, no wait that ran out."""
    b = Batch(32, "bf16", nh, kvh, hs, 64, [64 * 50 + 7, 3000, 500], [1, 500, 64])
    b.whole_bounds()
    sel = b.select(20, R)
    first = b.attend(sel, R, -0.2)
    busy = torch.randn(2048, 2048, device="cuda")
    for i in range(150):
        if i % 3 == 0:
            busy = busy @ busy * 1e-2
        out, lse = b.attend(sel, R, -0.2)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert int(b.error) == 0


@pytest.mark.parametrize("R", [1, 3, 16])
def test_sparse_attention_over_any_selection(R):
    """Selections of the caller's own: gaps of -1, nothing at all, pages behind the row, no own page."""
    b = Batch(10, "bf16", 8, 2, 128, 32, [32 * 12 + 9, 100, 0], [5, 64, 3], extra_rows=1)
    r = np.random.default_rng(3)
    sel = np.full((b.N, 2, 11), -1)
    for i in range(int(b.cum[-1])):
        s = int(np.searchsorted(b.cum, i, side="right")) - 1
        first = (i - b.cum[s]) // R * R
        n = (b.past[s] + min(first + R, b.q[s]) - 1) // 32 + 1
        for g in range(2):
            take = np.sort(r.permutation(n)[: r.integers(0, min(n, 11) + 1)])
            sel[i, g, np.sort(r.permutation(11)[: len(take)])] = take
    sel[0] = -1
    out, lse = b.attend(i32(sel), R)
    b.check(out, lse, sel, R)
    assert int(b.error) == 0


def test_sparse_attention_skips_and_reports_bad_entries():
    b = Batch(11, "fp16", 4, 2, 64, 16, [16 * 9 + 2, 40], [1, 2])
    good = np.array([[[0, 3, 9, -1], [1, 2, 9, -1]], [[0, 1, 2, -1]] * 2, [[-1, 0, 2, -1]] * 2])
    bad = np.array([[[0, 3, 9, 3], [1, 2, 9, 10]], [[0, 1, 2, 1 << 30], [0, 1, 2, -5]], [[-1, 0, 2, 2], [-1, 0, 2, 0]]])
    want = b.attend(i32(good))
    assert int(b.error) == 0
    got = b.attend(i32(bad))
    assert int(b.error) == pa.DEVERR_BAD_BLOCK
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    b.check(*want, good)


def test_sparse_attention_extreme_scores():
    """Large scores of either sign: the running maximum carries them, and one key takes all the weight."""
    b = Batch(12, "fp16", 4, 1, 64, 16, [16 * 40], [1], spread=4.0)
    b.whole_bounds()
    for scale in (3.0, -3.0):
        sel = b.select(12)
        out, lse = b.attend(sel, scale=scale)
        b.check(out, lse, sel.cpu().numpy(), scale=scale)


@pytest.mark.parametrize("R", [1, 3, 20])
def test_many_sequences_most_of_them_empty(R):
    """Sequences are found from a unit's number: through several levels of search, past runs of empty ones."""
    r = np.random.default_rng(9)
    B = 2600
    q = np.where(r.random(B) < 0.85, 0, r.integers(1, 7, B))
    q[0] = q[-1] = 0
    q[1234] = 45
    b = Batch(33, "bf16", 8, 2, 64, 16, r.integers(0, 120, B), q, extra_rows=5)
    got = b.bounds.clone()
    pa.update_page_bounds(b.key_cache, got, b.scale, *b.meta, num_tokens=b.N, error=b.error)
    keys = b.key_cache.float().cpu().numpy()
    assert np.array_equal(got.cpu().numpy(), ref.page_bounds(keys, np.zeros(got.shape), b.scale.cpu().numpy(), b.cum,
                                                             b.past, b.table))
    b.whole_bounds()
    sel = torch.full((b.N, 2, 5), -7, dtype=torch.int32, device="cuda")
    b.select(5, R, selected=sel)
    assert np.array_equal(sel.cpu().numpy(), b.want_selected(5, R))
    out, lse = b.attend(sel, R)
    b.check(out, lse, sel.cpu().numpy(), R)
    assert int(b.error) == 0


@pytest.mark.parametrize("R", [1, 32])
def test_offsets_past_32_bits(R):
    """A cache of more than 2^32 bytes and 2^31 values per tensor: pages at its end are where they should be."""
    kvh, hs, bs = 8, 128, 64
    small = Batch(34, "bf16", 32, kvh, hs, bs, [bs * 20 + 3], [33], extra_pages=0)
    small.whole_bounds()
    sel = small.select(8, R)
    want, wlse = small.attend(sel, R)
    blocks = (1 << 31) // (kvh * hs * bs) + 200
    big = [torch.empty(blocks, bs, kvh, hs, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    shift = blocks - small.blocks
    for x, y in zip(big, (small.key_cache, small.value_cache)):
        x[shift:] = y
    bounds = torch.zeros(blocks, kvh, 2, hs, dtype=torch.int8, device="cuda")
    table = i32(np.where(small.table >= 0, small.table + shift, -1))
    total = int(small.past[0] + small.q[0])
    pa.update_page_bounds(big[0], bounds, small.scale, i32([0, total]), i32([0]), table, num_tokens=total)
    assert torch.equal(bounds[shift:], small.bounds) and not bounds[:shift].any()
    kw = dict(num_heads=32, kv_num_heads=kvh, query_block=R)
    s2 = pa.select_pages(small.query, bounds, small.scale, *small.meta[:2], table, block_size=bs, top_k=8, **kw)
    assert torch.equal(s2, sel)
    lse = torch.empty_like(wlse)
    out = pa.sparse_paged_attention(small.query, *big, *small.meta[:2], table, sel, lse=lse, **kw)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_all_pages_selected_is_the_dense_attention():
    """With room for every page the sparse path is paged_attention on the same cache, within both roundings."""
    for dtype, R in (("fp16", 1), ("bf16", 8)):
        b = Batch(13, dtype, 8, 2, 128, 16, [100, 33, 0], [1, 20, 50])
        b.whole_bounds()
        sel = b.select(16, R)
        out, lse = b.attend(sel, R)
        kv = torch.zeros(b.N, 2 * 128, dtype=DT[dtype], device="cuda")
        lse2 = torch.empty_like(lse)
        dense = pa.paged_attention(b.query.contiguous(), kv, kv, b.key_cache, b.value_cache, *b.meta,
                                   i32(np.full(b.N, -1)), num_heads=8, kv_num_heads=2, lse=lse2)
        tol = 2 * torch.finfo(DT[dtype]).eps  # half a step each, and the weights' rounding (2^-11 of |V| < 4)
        assert ((out.double() - dense.double()).abs() <= tol * dense.double().abs() + 2.0 ** -9 * 4).all()
        assert ((lse - lse2).abs() <= 2e-4).all()


# ---- a step as it is used --------------------------------------------------------------------


def serving_step(s, n):
    """One step on packed rows: tables, rotation in place, cache write, bounds, selection, attention."""
    t = pa.build_block_tables(s["past"], s["q"], s["held"], s["table"], s["ring"], s["state"], block_size=s["bs"],
                              num_tokens=n, out=s.get("tables"))
    nh, kvh, hs = s["nh"], s["kvh"], s["hs"]
    q, k = s["rows"][:, : nh * hs], s["rows"][:, nh * hs: (nh + kvh) * hs]
    pa.qk_norm_rope(q, k, t.positions, num_heads=nh, kv_num_heads=kvh, q_norm_weight=s["w"], k_norm_weight=s["w"],
                    rotary_dim=hs, query_out=q, key_out=k)
    pa.paged_attention(s["rows"], None, None, s["kc"], s["vc"], t.cumulative_sequence_length, s["past"], s["table"],
                       t.slot_mapping, num_heads=nh, kv_num_heads=kvh, output=s["scratch"], workspace=s["ws"],
                       stages=pa.STAGE_PLAN | pa.STAGE_CACHE_WRITE)
    batch = (t.cumulative_sequence_length, s["past"], s["table"])
    pa.update_page_bounds(s["kc"], s["bounds"], s["scale"], *batch, num_tokens=n)
    sel = pa.select_pages(q, s["bounds"], s["scale"], *batch, num_heads=nh, kv_num_heads=kvh, block_size=s["bs"],
                          top_k=s["top_k"], query_block=s["R"])
    out = pa.sparse_paged_attention(q, s["kc"], s["vc"], *batch, sel, num_heads=nh, kv_num_heads=kvh,
                                    query_block=s["R"])
    return t, sel, out


def step_state(nh=8, kvh=2, hs=128, bs=16, B=5, blocks=120, cols=24, top_k=5, R=4, seed=0):
    r = np.random.default_rng(seed)
    s = dict(nh=nh, kvh=kvh, hs=hs, bs=bs, top_k=top_k, R=R)
    s["past"], s["held"], s["table"] = i32(np.zeros(B)), i32(np.zeros(B)), i32(np.full((B, cols), -1))
    s["ring"], s["state"] = i32(r.permutation(blocks)), i32([0, blocks])
    s["kc"], s["vc"] = (torch.zeros(blocks, bs, kvh, hs, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s["bounds"] = torch.zeros(blocks, kvh, 2, hs, dtype=torch.int8, device="cuda")
    s["scale"] = torch.full((kvh, hs), 0.03, device="cuda")
    s["w"] = torch.ones(hs, dtype=torch.bfloat16, device="cuda")
    return s


def rows_for(s, n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, (s["nh"] + 2 * s["kvh"]) * s["hs"], generator=g).to(torch.bfloat16).cuda()


def workspace_for(s, n):
    dims = pa.make_dims(n, len(s["past"]), s["hs"], s["kc"].shape[0], s["bs"], s["table"].shape[1], torch.bfloat16)
    return torch.zeros(pa.workspace_size(dims, s["nh"], s["kvh"]), dtype=torch.uint8, device="cuda")


def test_steps_together():
    """Prompts, then decode steps, a request leaving and another taking its pages; every step's output against the
    plain statements on the keys and values kept on the host."""
    s = step_state()
    nh, kvh, hs, bs = s["nh"], s["kvh"], s["hs"], s["bs"]
    past = np.zeros(5, int)
    history = [[np.zeros((0, kvh, hs))] * 2 for _ in range(5)]
    for step, q in enumerate([[100, 37, 0, 64, 1], [1, 1, 50, 1, 1], [1, 1, 1, -1, 1], [4, 4, 0, 90, 4], [1] * 5]):
        q = np.array(q)
        n = int(np.maximum(q, 0).sum())
        s["q"], s["rows"] = i32(q), rows_for(s, n, step)
        raw = f64(s["rows"])
        s["scratch"] = torch.empty(n, nh * hs, dtype=torch.bfloat16, device="cuda")
        s["ws"] = workspace_for(s, n)
        t, sel, out = serving_step(s, n)
        assert int(t.error) == 0 and pa.read_device_error(s["ws"]) == 0
        cum = t.cumulative_sequence_length.cpu().numpy()
        # the rotated rows are what the statement says, and what the cache holds
        p = t.positions.cpu().numpy()
        y, size = ref.norm_rope(raw[:, : (nh + kvh) * hs].reshape(n, nh + kvh, hs), np.ones(hs), float(np.float32(1e-6)),
                                p, hs, 1e4, False)
        got = f64(s["rows"])[:, : (nh + kvh) * hs].reshape(y.shape)
        assert (np.abs(got - y) <= rotate_bound(y, size, "bf16")).all()
        for b in range(5):
            if q[b] < 0:
                history[b] = [np.zeros((0, kvh, hs))] * 2
            elif q[b]:
                rows = slice(cum[b], cum[b + 1])
                history[b] = [np.concatenate([history[b][0], got[rows, nh:]]),
                              np.concatenate([history[b][1], raw[rows, (nh + kvh) * hs:].reshape(-1, kvh, hs)])]
        table, kc, vc = s["table"].cpu().numpy(), f64(s["kc"]), f64(s["vc"])
        kc2, vc2 = np.zeros_like(kc), np.zeros_like(vc)
        want_bounds = s["bounds"].cpu().numpy().astype(int)
        for b in range(5):
            for page in range(-(-len(history[b][0]) // bs)):
                part = [h[page * bs: (page + 1) * bs] for h in history[b]]
                kc2[table[b, page], : len(part[0])], vc2[table[b, page], : len(part[1])] = part
                c = ref.key_codes(part[0], s["scale"].cpu().numpy())
                want_bounds[table[b, page], :, 0], want_bounds[table[b, page], :, 1] = c.min(0), c.max(0)
                assert np.array_equal(kc[table[b, page], : len(part[0])], part[0])
        assert np.array_equal(s["bounds"].cpu().numpy(), want_bounds)
        lens = np.where(q < 0, 0, past)
        want = ref.select_pages(s["rows"].float().cpu().numpy()[:, : nh * hs].reshape(n, nh, hs), want_bounds,
                                s["scale"].cpu().numpy(), cum, lens, table, kvh, bs, s["top_k"], s["R"], 1, 1)
        assert np.array_equal(sel.cpu().numpy(), want)
        o, _, size, mag = ref.sparse_attention(got[:, :nh], kc2, vc2, cum, lens, table, want, hs ** -0.5, s["R"])
        # (half a step of bf16 is 2^-8 of the value)
        bound = 2.0 ** -8 * np.abs(o) * 1.01 + size * (2.0 ** -16 + mag[..., None] * (hs + 8) * 2.0 ** -22 + 2.0 ** -16)
        off = np.abs(f64(out).reshape(o.shape) - o)
        assert float((off / bound).max()) <= 1
        past = np.where(q < 0, 0, past + q)
        s["past"] = i32(past)
        s["held"], s["state"] = t.blocks_held, t.free_state


def test_captured_step_replays():
    """A decode step as a CUDA graph on a side stream: replays on new rows and lengths give what the calls give."""
    s = step_state(seed=4)
    n = 5
    s["q"], s["past"] = i32([90, 40, 64, 17, 1]), i32(np.zeros(5))
    first = rows_for(s, 212, 0)
    s["rows"], s["scratch"] = first, torch.empty(212, s["nh"] * s["hs"], dtype=torch.bfloat16, device="cuda")
    s["ws"] = workspace_for(s, 212)
    t, _, _ = serving_step(s, 212)
    s["held"], s["state"], s["past"] = t.blocks_held.clone(), t.free_state.clone(), s["q"].clone()
    s["q"] = i32([1] * 5)
    s["rows"], s["scratch"] = rows_for(s, n, 1), torch.empty(n, s["nh"] * s["hs"], dtype=torch.bfloat16, device="cuda")
    s["ws"] = workspace_for(s, n)
    keep = {k: v.clone() for k, v in s.items() if torch.is_tensor(v)}

    def reset(src):
        for k, v in src.items():
            s[k].copy_(v)

    def advance(t):
        s["past"] += s["q"]
        s["held"].copy_(t.blocks_held)
        s["state"].copy_(t.free_state)

    eager = []
    for i in range(20):  # crosses page ends
        s["rows"].copy_(rows_for(s, n, 10 + i))
        t, sel, out = serving_step(s, n)
        eager.append((sel.clone(), out.clone(), t.slot_mapping.clone()))
        advance(t)
    reset(keep)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        serving_step(s, n)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        t, sel, out = serving_step(s, n)
        advance(t)
    reset(keep)
    for i in range(20):
        s["rows"].copy_(rows_for(s, n, 10 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(sel, eager[i][0]) and torch.equal(out, eager[i][1])
        assert torch.equal(t.slot_mapping, eager[i][2])


def test_calls_on_two_streams_at_once():
    """The operators share no state: two batches on two streams give what each gives alone."""
    batches = []
    for seed, R in ((20, 1), (21, 16)):
        b = Batch(seed, "fp16", 16, 2, 128, 16, [1500, 3000, 700], [1, 33, 2])
        b.whole_bounds()
        sel = b.select(20, R)
        batches.append((b, R, sel, *b.attend(sel, R)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    got = [[], []]
    for _ in range(10):
        for k, (b, R, *_rest) in enumerate(batches):
            with torch.cuda.stream(streams[k]):
                sel = b.select(20, R)
                got[k].append((sel, *b.attend(sel, R)))
    torch.cuda.synchronize()
    for k, (_, _, sel, out, lse) in enumerate(batches):
        for s2, o2, z2 in got[k]:
            assert torch.equal(s2, sel) and torch.equal(o2, out) and torch.equal(z2, lse)


class _NoFast:
    """The compiled calls as they answer anything unusual."""

    def __getattr__(self, name):
        return lambda *a: None


def test_both_ways_into_the_library_agree(monkeypatch):
    """The compiled calls and the Python code behind them: the same results, types and shapes."""
    from varlen_paged_kv_gb300 import step

    def results():
        out = []
        for dtype, R in (("fp16", 1), ("bf16", 5)):
            b = Batch(41, dtype, 8, 2, 128, 16, [300, 45], [1, 12], extra_rows=2, wide=256)
            b.whole_bounds()
            sel = b.select(6, R)
            lse = torch.zeros(b.N, 8, device="cuda")
            o = pa.sparse_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, sel, num_heads=8, kv_num_heads=2,
                                          scale=0.11, query_block=R, lse=lse, error=b.error)
            n = int(b.cum[-1])
            w = torch.ones(128, dtype=DT[dtype], device="cuda")
            k = b.rows[:, 1024:]
            turned = pa.qk_norm_rope(b.query, k, i32(np.arange(b.N)), num_heads=8, kv_num_heads=2, q_norm_weight=w,
                                     eps=1e-5, rotary_dim=64, theta=5e5, interleaved=R == 1)
            out += [b.bounds, sel[:n], o[:n], lse[:n], b.error, *turned]
        a = table_state(np.random.default_rng(6), 30, 16, 20, 200, 40, 0.2)
        t, dev = run_tables(*a, 16, 700)
        return out + list(t) + dev

    fast = results()
    assert step._fast is not None
    monkeypatch.setattr(step, "_fast", _NoFast())
    for x, y in zip(fast, results()):
        assert x.dtype == y.dtype and x.shape == y.shape and x.is_contiguous() and torch.equal(x, y)


def test_refusals_say_what_was_wrong():
    b = Batch(42, "fp16", 4, 2, 64, 16, [100], [2])
    kw = dict(num_heads=4, kv_num_heads=2)
    sel = b.select(4)
    with pytest.raises(TypeError, match="selected must be int32"):
        pa.sparse_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, sel.long(), **kw)
    with pytest.raises(TypeError, match="value_cache"):
        pa.sparse_paged_attention(b.query, b.key_cache, b.value_cache.bfloat16(), *b.meta, sel, **kw)
    with pytest.raises(ValueError, match="selected must be a contiguous"):
        pa.sparse_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, sel.transpose(0, 1), **kw)
    with pytest.raises(ValueError, match="lse"):
        pa.sparse_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, sel, lse=torch.zeros(2, 3).cuda(), **kw)
    with pytest.raises(ValueError, match="batch_size"):
        pa.select_pages(b.query, b.bounds, b.scale, b.meta[0][:1], *b.meta[1:], block_size=16, top_k=4, **kw)
    with pytest.raises(pa.PagedAttentionError, match="INVALID_ARGUMENT"):
        pa.select_pages(b.query, b.bounds, b.scale, *b.meta, block_size=16, top_k=1, **kw)
    with pytest.raises(pa.PagedAttentionError, match="UNSUPPORTED"):
        pa.select_pages(b.query, b.bounds, b.scale, *b.meta, block_size=24, top_k=4, **kw)
    with pytest.raises(pa.PagedAttentionError, match="INVALID_ARGUMENT"):  # rows that do not start on 16 bytes
        wide = torch.zeros(2, 300, dtype=torch.float16, device="cuda")
        pa.select_pages(wide[:, :256], b.bounds, b.scale, *b.meta, block_size=16, top_k=4, **kw)
    with pytest.raises(ValueError, match="key must be"):
        pa.qk_norm_rope(b.query, b.query, i32([0, 1]), **kw)
    with pytest.raises(pa.PagedAttentionError, match="UNSUPPORTED"):
        pa.qk_norm_rope(b.query, b.query[:, :128], i32([0, 1]), rotary_dim=8, **kw)
    with pytest.raises(TypeError, match="int8"):
        pa.update_page_bounds(b.key_cache, b.bounds.int(), b.scale, *b.meta, num_tokens=2)
    with pytest.raises(ValueError, match="block_table"):
        pa.build_block_tables(b.meta[1], b.meta[1], b.meta[1], b.meta[2][:0], b.meta[1], i32([0, 0]), block_size=16,
                              num_tokens=4)
    with pytest.raises(ValueError, match="negative"):
        pa.build_block_tables(b.meta[1], b.meta[1], b.meta[1], b.meta[2], b.meta[1], i32([0, 0]), block_size=16,
                              num_tokens=-1)
    torch.cuda.synchronize()


def test_explicit_stream_argument():
    b = Batch(22, "fp16", 4, 2, 64, 16, [300], [2])
    b.whole_bounds()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(5):
        # freed blocks of the current stream, still in use there, are not what the side stream writes to
        junk = torch.zeros(2, 2, 5, dtype=torch.int32, device="cuda")
        for _ in range(20):
            busy = busy @ busy * 1e-3
        seen = junk.clone()
        del junk
        sel = b.select(5, stream=side)
        out = pa.sparse_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, sel, num_heads=4, kv_num_heads=2,
                                        stream=side)
        side.synchronize()
        assert np.array_equal(sel.cpu().numpy(), b.want_selected(5))
        want, lse = b.attend(sel)
        assert torch.equal(out, want) and (seen == 0).all()
        b.check(want, lse, sel.cpu().numpy())
    q, k = b.query.contiguous(), b.query[:, :128].contiguous()
    side.wait_stream(torch.cuda.current_stream())
    pos = i32([5, 6])
    torch.cuda.synchronize()
    on = pa.qk_norm_rope(q, k, pos, num_heads=4, kv_num_heads=2, rotary_dim=64, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(on, pa.qk_norm_rope(q, k, pos, num_heads=4, kv_num_heads=2,
                                                                     rotary_dim=64)))
