"""Attention with capped and biased scores, windows, documents and prefixes against its plain statement in 64 bits
(pool_reference), within bounds derived from the roundings."""
import numpy as np
import pytest
import torch

import pool_reference as ref
import varlen_paged_kv_gb300 as pa
from test_step_gpu import DT, Batch, f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.fail("CUDA is required for the gpu tests")
    from varlen_paged_kv_gb300 import build
    build.build()


class Rules:
    """A call's rules, as the tensors of the call and as the plain statement takes them."""

    def __init__(self, b, softcap=0.0, bias=False, window=0, documents=0, prefix=0, seed=0, scale=0.0, bound=None):
        r = np.random.default_rng(seed + 1)
        self.softcap, self.window, self.scale, self.bound = softcap, window, scale, bound
        self.slopes = (2.0 ** (-8 * np.arange(1, b.nh + 1) / b.nh)).astype(np.float32) if bias else None
        self.first = self.prefix = None
        if documents:
            first = []
            for s in range(len(b.past)):
                total = int(b.past[s] + b.q[s])
                cuts = np.concatenate([[0], np.cumsum(r.integers(1, 2 * documents, 2 + 3 * total // documents))])
                pos = int(b.past[s]) + np.arange(b.q[s])
                start = cuts[np.searchsorted(cuts, pos, side="right") - 1]
                first.append(np.where(r.random(b.q[s]) < 0.1, total + r.integers(0, 3), start))
            self.first = np.concatenate(first + [np.full(b.N - int(b.cum[-1]), -4)])
        if prefix:
            self.prefix = r.integers(-3, prefix + 1, len(b.past))

    def call(self, b, **kw):
        t = lambda a: None if a is None else i32(a)  # noqa: E731
        lse = torch.full((b.N, b.nh), 5.0, device="cuda")
        out = torch.full((b.N, b.nh * b.hs), 5.0, dtype=DT[b.dtype], device="cuda")
        kw = dict(output=out, lse=lse, error=b.error, max_query_len=self.bound if self.bound is not None else 0) | kw
        pa.biased_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, num_heads=b.nh, kv_num_heads=b.kvh,
                                  scale=self.scale, softcap=self.softcap,
                                  slopes=None if self.slopes is None else torch.from_numpy(self.slopes).cuda(),
                                  window=self.window, first_keys=t(self.first), prefix_lens=t(self.prefix), **kw)
        return kw["output"], kw["lse"]

    def check(self, b, out, lse, key_cache=None, value_cache=None, rows=slice(None)):
        sc = float(np.float32(self.scale)) if self.scale else b.hs ** -0.5
        o, z, size, mag, far = ref.biased_attention(
            f64(b.query).reshape(b.N, b.nh, b.hs), f64(b.key_cache if key_cache is None else key_cache),
            f64(b.value_cache if value_cache is None else value_cache), b.cum, b.past, b.table, sc, self.softcap,
            self.slopes, self.window, self.first, self.prefix)
        n = int(b.cum[-1])
        got, gz = f64(out).reshape(o.shape), f64(lse)
        assert (got[n:] == 5).all() and (gz[n:] == 5).all()  # rows behind the last sequence
        o, z, size, mag, far, got, gz = (x[:n][rows] for x in (o, z, size, mag, far, got, gz))
        # a score's error: hs products summed in fp32 (at most one unit of 2^-23 of the sum of magnitudes a step), the
        # scale; of the cap the hyperbolic tangent, 2^-21 of it (an exponential, a sum, a reciprocal and its own
        # rounding, 2^-23 each), of the bias three roundings; the exponent's argument and the exponential, 2^-21 each
        # of the score's size; each weight enters P V rounded to fp16 (half a step, 2^-11) or as two bf16 terms
        # (2^-16); sums over the keys and the merge of partial results 2^-18; then one rounding to T
        finite = np.where(np.isfinite(z), np.abs(z), 0)
        delta = (mag * (b.hs + 8) * 2.0 ** -23 + self.softcap * 2.0 ** -21 + far * 2.0 ** -22 +
                 2.0 ** -21 * (1 + finite + self.softcap))
        weight = 2.0 ** -11 if b.dtype == "fp16" else 2.0 ** -16
        eps = torch.finfo(DT[b.dtype]).eps / 2
        tiny = 2.0 ** -25 if b.dtype == "fp16" else 0.0
        bound = eps * np.abs(o) * (1 + 2.0 ** -7) + size * (weight + 2 * delta[..., None] + 2.0 ** -17) + tiny
        assert (np.abs(got - o) <= bound).all(), (np.abs(got - o) / bound).max()
        none = np.isneginf(z)
        assert np.array_equal(none, np.isneginf(gz))
        assert (np.abs(gz[~none] - z[~none]) <= (delta + 2.0 ** -17)[~none]).all()
        assert (got[none] == 0).all()


SHAPES = [(8, 2, 64), (4, 4, 128), (16, 2, 256), (8, 1, 128), (7, 1, 64), (14, 2, 64), (32, 8, 128), (20, 1, 64)]
KINDS = [dict(), dict(softcap=20.0), dict(bias=True), dict(window=50), dict(documents=40), dict(prefix=90),
         dict(softcap=3.0, bias=True, window=70, documents=60, prefix=60)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("nh,kvh,hs", SHAPES)
def test_biased_attention(nh, kvh, hs, kind, dtype):
    """Decode rows, drafts and prompts in one batch, rows that see nothing, rows of no sequence."""
    seed = nh * 100 + hs + kind
    bs = [16, 32, 48, 64, 256][seed % 5]
    b = Batch(seed, dtype, nh, kvh, hs, bs, past=[0, 63, 200, 31, 0, 500, 17], q=[1, 2, 1, 60, 0, 150, 3], extra_rows=2,
              wide=2 * kvh * hs)
    rules = Rules(b, seed=seed, **KINDS[kind])
    out, lse = rules.call(b)
    assert int(b.error) == 0
    rules.check(b, out, lse)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nh,kvh,hs,bs,past,q,kw", [
    (8, 8, 64, 16, [700], [1], dict(softcap=50.0)),                        # one row, many shares
    (32, 8, 128, 64, [4000, 1], [1, 1], dict(bias=True)),                  # a long row beside a short one
    (4, 1, 128, 16, [63, 64, 65, 127, 128, 0], [1] * 6, dict(window=64)),  # windows at the ends of tiles
    (4, 1, 128, 16, [63, 64, 65, 127, 128, 0], [1] * 6, dict(window=1)),
    (16, 2, 256, 32, [3000, 10, 800], [2, 1, 2], dict(softcap=30.0, window=1000)),
    (8, 2, 128, 256, [900], [4], dict(prefix=3000)),                       # a prefix past the end
    (8, 2, 64, 16, [100] * 400, [1] * 400, dict(documents=30)),            # more sequences than a block's threads
    (8, 2, 64, 16, [30] * 70, [16] * 70, dict(softcap=10.0, bound=16)),    # 64 rows each, the bound given
    (130, 1, 64, 16, [100, 40], [3, 1], dict(softcap=10.0, bias=True)),    # a group of more than a tile's rows
    (64, 1, 64, 16, [5000], [1], dict(window=3000)),                       # a wide group: clusters over the keys
    (4, 2, 128, 16, [9000], [40], dict(softcap=20.0, prefix=9020)),        # few rows, many keys
    (1, 1, 128, 48, [0, 300], [257, 130], dict(documents=50, prefix=100)),
    (6, 2, 256, 16, [0, 77], [90, 300], dict(softcap=5.0, bias=True)),
    (2, 2, 64, 16, [0], [600], dict(window=100, prefix=80)),
    (32, 8, 128, 64, [2500, 100], [600, 300], dict(softcap=30.0, bias=True, documents=900, prefix=200)),
    (16, 4, 128, 256, [0] * 40, [70] * 40, dict(window=33, softcap=30.0)),
    (16, 2, 256, 32, [900, 5, 300, 0], [5, 4, 8, 1], dict(softcap=30.0, window=400, bound=8)),  # 64 rows of a tile
    (16, 2, 256, 16, [3000], [7], dict(bias=True, documents=500, bound=7)),
    (3, 1, 256, 48, [700, 64], [21, 11], dict(prefix=800, bound=21))])
def test_biased_attention_at_the_edges(nh, kvh, hs, bs, past, q, kw, dtype):
    b = Batch(nh + len(past), dtype, nh, kvh, hs, bs, past, q)
    rules = Rules(b, seed=3, **kw)
    out, lse = rules.call(b)
    assert int(b.error) == 0
    rules.check(b, out, lse)
    # the same call again gives the same bits
    again, z = rules.call(b)
    assert torch.equal(out, again) and torch.equal(lse, z)


@pytest.mark.parametrize("nh,kvh,q", [(8, 2, 1), (8, 2, 40)])
def test_scores_from_tiny_to_saturated(nh, kvh, q):
    """Caps that bend nothing, and caps that every score is far beyond, both signs of the scale."""
    b = Batch(9, "fp16", nh, kvh, 128, 16, [300, 20], [q, q], spread=2.0)
    for scale, cap in ((1e-4, 50.0), (0.088, 1000.0), (0.088, 0.5), (1.0, 30.0), (-0.1, 20.0), (5.0, 1.0), (-0.05, 0.0)):
        rules = Rules(b, softcap=cap, scale=scale)
        out, lse = rules.call(b)
        rules.check(b, out, lse)


def test_pages_that_a_window_left_behind_are_not_looked_up():
    for q in (1, 30):
        b = Batch(21, "bf16", 8, 2, 128, 16, [500, 90], [q, q])
        rules = Rules(b, window=64)
        want = rules.call(b)
        for s in range(2):
            gone = max(0, (int(b.past[s]) - 63) // 16)
            b.table[s, :gone] = [-1, 1 << 30, b.blocks][s % 3]
        b.meta = (*b.meta[:2], i32(b.table))
        got = rules.call(b)
        assert int(b.error) == 0
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("q", [1, 30])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -65504.0])
def test_what_unseen_keys_hold_reaches_nothing(q, fill):
    """Keys before a window or a document's start, in pages that are read for their later keys."""
    b = Batch(22, "fp16", 8, 2, 64, 64, [200, 90], [q, q])
    rules = Rules(b, window=70)
    rules.first = np.concatenate([np.full(q, 150), np.full(q, 80)])
    out, lse = rules.call(b)
    kc, vc = b.key_cache.clone(), b.value_cache.clone()
    for s in range(2):
        for t in range(max([150, 80][s], int(b.past[s]) - 69)):
            kc[b.table[s, t // 64], t % 64] = fill
            vc[b.table[s, t // 64], t % 64] = fill
    b.key_cache, b.value_cache = kc, vc
    got, z = rules.call(b)
    assert torch.equal(out, got) and torch.equal(lse, z)


@pytest.mark.parametrize("q", [1, 40])
def test_keys_and_queries_of_nan(q):
    b = Batch(23, "fp16", 8, 2, 64, 16, [200, 90], [q, q])
    b.key_cache[b.table[0, 3], 5, 0] = float("nan")
    b.query[q] = float("nan")
    for kw in (dict(), dict(softcap=9.0), dict(bias=True)):
        out, lse = Rules(b, **kw).call(b)
        o, z = out.view(-1, 8, 64), lse
        assert torch.isnan(o[:q, :4]).all() and torch.isnan(z[:q, :4]).all()       # rows that see the key
        assert torch.isfinite(o[:q, 4:]).all() and torch.isfinite(z[:q, 4:]).all()
        assert torch.isnan(o[q]).all() and torch.isfinite(o[q + 1:]).all()


def test_bad_batches_and_pages_are_reported():
    for q in (1, 30):
        b = Batch(24, "fp16", 8, 2, 64, 16, [200, 90, 40], [q, q, q])
        rules = Rules(b)
        others = np.r_[0: q, 2 * q: 3 * q]  # (what the shares of the work are, their last bits depend on)
        bad = b.table.copy()
        bad[1, 2] = b.blocks
        b.meta = (*b.meta[:2], i32(bad))
        out, lse = rules.call(b)
        assert int(b.error) == pa.DEVERR_BAD_BLOCK
        rules.check(b, out, lse, rows=others)
        b.error.zero_()
        b.meta = (b.meta[0], i32([200, -1, 40]), i32(b.table))
        out, lse = rules.call(b)
        assert int(b.error) == pa.DEVERR_BAD_BATCH
        rules.check(b, out, lse, rows=others)
        assert (out[q: 2 * q] == 5).all() and (lse[q: 2 * q] == 5).all()
        b.error.zero_()
        b.meta = (i32(b.cum), i32(b.past), i32(b.table))
        if q > 1:  # longer than the bound that the call was given
            rules.bound = 4
            out, _ = rules.call(b)
            assert int(b.error) == pa.DEVERR_BAD_BATCH and (out == 5).all()


def test_plain_rules_are_the_dense_attention():
    for dtype in ("fp16", "bf16"):
        b = Batch(25, dtype, 8, 2, 128, 16, [300, 64, 0], [1, 3, 200])
        rules = Rules(b)
        out, lse = rules.call(b)
        dense_lse = torch.empty_like(lse)
        n = b.N
        ws = torch.zeros(pa.workspace_size(pa.make_dims(n, 3, 128, b.blocks, 16, b.table.shape[1], DT[dtype]), 8, 2),
                         dtype=torch.uint8, device="cuda")
        dense = pa.paged_attention(b.query.contiguous(), torch.zeros(n, 256, dtype=DT[dtype], device="cuda"),
                                   torch.zeros(n, 256, dtype=DT[dtype], device="cuda"), b.key_cache.clone(),
                                   b.value_cache.clone(), *b.meta, i32([-1] * n), num_heads=8, kv_num_heads=2,
                                   lse=dense_lse, workspace=ws)
        # half a step each, and the weights' rounding (2^-11 of |V| < 4.5)
        tol = 2 * torch.finfo(DT[dtype]).eps
        assert ((out.double() - dense.double()).abs() <= tol * dense.double().abs() + 2.0 ** -9 * 4.5).all()
        assert (lse - dense_lse).abs().max() < 1e-4


def test_offsets_past_32_bits():
    """A pool of more than 2^31 values and sequences at its end."""
    blocks, bs, kvh, hs = 36000, 256, 4, 64
    kc = torch.zeros(blocks, bs, kvh, hs, dtype=torch.float16, device="cuda")
    vc = torch.zeros(blocks, bs, kvh, hs, dtype=torch.float16, device="cuda")
    g = torch.Generator().manual_seed(1)
    used = [35999, 35000, 34001, 2]
    for p in used:
        kc[p], vc[p] = (torch.randn(bs, kvh, hs, generator=g).half().cuda() for _ in range(2))
    for q in (1, 40):
        b = Batch(26, "fp16", 8, 4, 64, 256, [900 - q], [q])
        b.table = np.array([used])
        b.meta = (*b.meta[:2], i32(b.table))
        small = np.arange(4)[None]
        b.key_cache, b.value_cache, b.blocks = kc, vc, blocks
        rules = Rules(b, softcap=20.0)
        out, lse = rules.call(b)
        assert int(b.error) == 0
        b.table = small
        rules.check(b, out, lse, kc[used], vc[used])


def test_captured_calls_on_two_streams_at_once():
    """Two graphs with workspaces of their own and calls between them."""
    made = []
    for seed, q in ((31, 1), (32, 3), (33, 70)):
        b = Batch(seed, "bf16", 8, 2, 128, 16, [700, 30, 90], [q, 1, q])
        rules = Rules(b, softcap=30.0, window=400)
        made.append((b, rules, rules.call(b)))
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream() for _ in made], [], []
    for (b, rules, _), s in zip(made, streams):
        with torch.cuda.stream(s):
            rules.call(b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        t = {k: torch.zeros_like(v) for k, v in zip(("output", "lse"), made[len(graphs)][2])}
        slopes = rules.slopes
        assert slopes is None
        with torch.cuda.graph(graph, stream=s):
            rules.call(b, **t)
        graphs.append(graph)
        outs.append(t)
    for _ in range(5):
        for t in outs:
            t["output"].zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for t, (_, _, want) in zip(outs, made):
            assert torch.equal(t["output"], want[0]) and torch.equal(t["lse"], want[1])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("past,q,kw,longest", [
    ([60], [3], dict(), 4),                             # a cluster's item
    ([60, 900, 0], [3, 4, 2], dict(softcap=20.0), 0),   # whole items and pieces that are merged
    ([9000] * 3, [4, 4, 1], dict(bias=True), 4),
    ([60, 5], [70, 200], dict(softcap=9.0), 0),         # tiles
    ([2000], [12], dict(prefix=30), 0),                 # a cluster's tile
    ([100, 30], [90, 64], dict(documents=25), 0)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them_only(past, q, kw, longest, fill, dtype):
    nh, kvh, hs = 8, 2, 128
    b = Batch(41, dtype, nh, kvh, hs, 16, past, q)
    rules = Rules(b, seed=5, bound=longest or None, **kw)
    for s in range(len(past)):  # a key among the new rows, seen by the later ones of its block alone
        t = past[s] + q[s] // 2
        b.value_cache[b.table[s, t // 16], t % 16, 1] = fill
    out, lse = rules.call(b)
    assert int(b.error) == 0
    sc = hs ** -0.5
    with np.errstate(invalid="ignore"):
        o, z, _, _, _ = ref.biased_attention(f64(b.query).reshape(b.N, nh, hs), f64(b.key_cache), f64(b.value_cache), b.cum,
                                             b.past, b.table, sc, rules.softcap, rules.slopes, rules.window, rules.first,
                                             rules.prefix)
    got = f64(out).reshape(o.shape)
    clean = np.isfinite(o).all((1, 2))
    assert clean.any() and not clean.all()
    with np.errstate(invalid="ignore"):
        rules.check(b, out, lse, rows=np.flatnonzero(clean))
    # a weight may be 0 in 32 bits where it is not in 64, and 0 times infinity is NaN
    far = ~clean
    assert np.array_equal(np.isfinite(got[far]), np.isfinite(o[far]))
    assert (np.isposinf(got[far]) | np.isnan(got[far]) | np.isfinite(got[far])).all()
    assert (np.abs(f64(lse)[~np.isneginf(z)] - z[~np.isneginf(z)]) < 1e-3).all()


LONG = [(8, 2, 128, 64, [100, 700, 0], [600, 3, 520], dict(softcap=20.0, bias=True, documents=300, prefix=50)),
        (16, 16, 64, 16, [0], [2100], dict(window=200)),                 # one head a group
        (16, 2, 256, 32, [300, 2000], [256, 300], dict(prefix=5000)),
        (8, 2, 128, 48, [30], [515], dict(documents=60))]


@pytest.mark.parametrize("values", ["plain", "large", "tiny", "inf", "small heads"])
@pytest.mark.parametrize("nh,kvh,hs,bs,past,q,kw", LONG)
def test_long_sequences_of_all_sorts_of_values(nh, kvh, hs, bs, past, q, kw, values):
    """Values far apart, large and tiny ones, one that is not finite."""
    b = Batch(61, "bf16", nh, kvh, hs, bs, past, q)
    if values == "large":  # one that is larger than all others
        b.value_cache[b.table[0, 1], 2, 0, 3] = 300.0
    elif values == "tiny":
        b.value_cache.mul_(1e-7)
    elif values == "inf":
        b.value_cache[b.table[0, (past[0] + q[0] - 1) // bs], 0, 0] = float("inf")
    elif values == "small heads":  # the heads far apart
        b.value_cache[:, :, 0] *= 2.0 ** -10
        b.value_cache[:, :, -1] *= 60.0 if kvh > 1 else 1.0
    rules = Rules(b, seed=7, **kw)
    out, lse = rules.call(b)
    assert int(b.error) == 0
    if values == "inf":
        o = f64(out).reshape(b.N, nh, hs)
        first = past[0] + q[0] - 1
        first -= first % bs  # the key that is not finite; the rows before it do not see it unless their prefix does
        if "prefix" not in kw:
            before = np.arange(max(0, first - past[0] - 1))
            rules.check(b, out, lse, rows=before)
        assert not np.isfinite(o).all()
    else:
        rules.check(b, out, lse)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("past,q,kw", [([700, 3, 90], [1, 4, 2], dict()), ([300, 0], [120, 200], dict(softcap=20.0)),
                                       ([200], [150], dict(prefix=260)), ([2000], [30], dict())])
def test_slopes_of_either_sign(past, q, kw, dtype):
    """A negative slope favours the farthest keys."""
    b = Batch(51, dtype, 8, 2, 128, 32, past, q)
    rules = Rules(b, seed=7, bias=True, **kw)
    rules.slopes[::2] *= -1
    rules.slopes[3] = 0
    out, lse = rules.call(b)
    assert int(b.error) == 0
    rules.check(b, out, lse)


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_values_that_are_not_finite_in_many_short_sequences(fill):
    """Several whole sequences for each block, with rows to compute again in all of them."""
    test_values_that_are_not_finite_reach_the_rows_that_see_them_only([30] * 300, [3] * 300, dict(softcap=20.0), 4, fill,
                                                                      "fp16")


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("past,q,longest", [([90], [2], 2), ([90, 9000, 5], [2, 1, 1], 2), ([40], [60], 0)])
def test_one_key_of_nan_makes_the_rows_nan_that_see_it(past, q, longest, where):
    """A cluster's item, whole items and merged pieces, a tile's."""
    b = Batch(61, "fp16", 8, 2, 128, 16, past, q)
    rules = Rules(b, seed=2, bound=longest or None, softcap=20.0, window=80 if where == "first" else 0)
    t = {"first": 20, "middle": 37, "last": past[0]}[where]  # (in a window of 80 the first rows' first key is 11 or more)
    if where == "first" and past[0] == 90:
        t = 11  # the first key of row 0, not seen by row 1
    b.key_cache[b.table[0, t // 16], t % 16, 1] = float("nan")
    out, lse = rules.call(b)
    assert int(b.error) == 0
    got, z = f64(out).reshape(b.N, 8, 128), f64(lse)
    for j in range(b.N):
        mine = j < q[0]
        pos = past[0] + j
        sees = mine and t <= pos and (not rules.window or t > pos - rules.window)
        assert np.isnan(got[j, 4:]).all() if sees else np.isfinite(got[j]).all(), j
        assert np.isnan(z[j, 4:]).all() if sees else np.isfinite(z[j]).all(), j
        assert np.isfinite(got[j, :4]).all() and np.isfinite(z[j, :4]).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("softcap,size", [(50.0, 1.0), (50.0, 2.5), (50.0, 5.0), (50.0, 40.0), (160.0, 30.0), (400.0, 2.0), (400.0, 60.0),
                                          (3000.0, 200.0), (1e30, 1.0)])
def test_caps_small_and_large_against_their_scores(softcap, size, dtype):
    """Every form of the cap: all scores near zero, some way up, most of them at the cap, caps that are none."""
    for hs, past, q, bound in ((128, [70, 0, 300], [1, 200, 150], 0), (256, [130, 20], [60, 1], 0), (64, [400], [2], 2)):
        b = Batch(71, dtype, 8, 2, hs, 32, past, q)
        b.query[::2] *= size
        b.query[1::4] *= -size
        for kw in (dict(), dict(bias=True, prefix=150)):
            rules = Rules(b, seed=9, softcap=softcap, bound=bound or None, **kw)
            out, lse = rules.call(b)
            assert int(b.error) == 0
            rules.check(b, out, lse)
