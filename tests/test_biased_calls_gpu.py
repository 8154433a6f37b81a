"""Calls of the biased attention that the documentation allows and that once went wrong, or that no other test makes,
against the plain statement in 64 bits (pool_reference)."""
import numpy as np
import pytest
import torch

import pool_reference as ref
import varlen_paged_kv_gb300 as pa
from test_biased_gpu import Rules
from test_step_gpu import DT, Batch, _NoFast, f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.fail("CUDA is required for the gpu tests")
    from varlen_paged_kv_gb300 import build
    build.build()


# ---- pages that no row sees, between pages that some rows of a block see -----------------------


def _between_documents(nh, kvh, hs, past, q, pad, dtype="bf16"):
    """One sequence of a document, `pad` rows that see nothing, and another document; the pages wholly inside the padding."""
    b = Batch(81, dtype, nh, kvh, hs, 16, [past], [q])
    rules = Rules(b)
    at = (q - pad) // 2
    rules.first = np.concatenate([np.zeros(at), np.full(pad, past + q), np.full(q - at - pad, past + at + pad)]).astype(int)
    unseen = np.arange(-(-(past + at) // 16), (past + at + pad) // 16)
    assert len(unseen)
    return b, rules, unseen


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nh,kvh,hs,past,q,pad", [
    (2, 2, 64, 0, 120, 60), (2, 2, 128, 30, 126, 70), (2, 2, 256, 0, 128, 50),  # one block of 128 rows of a head
    (2, 2, 128, 500, 100, 40), (4, 2, 64, 3000, 60, 45),                        # few blocks: clusters over the keys
    (130, 1, 64, 20, 100, 60)])                                                 # a group of more than a tile's rows
def test_pages_between_documents_may_be_anything(nh, kvh, hs, past, q, pad, dtype):
    b, rules, unseen = _between_documents(nh, kvh, hs, past, q, pad, dtype)
    want = rules.call(b)
    rules.check(b, *want)
    for fill in (-1, 1 << 30, b.blocks, -(1 << 31)):
        table = b.table.copy()
        table[0, unseen] = fill
        b.meta = (*b.meta[:2], i32(table))
        got = rules.call(b)
        assert int(b.error) == 0
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("nh,kvh,hs,past,q,pad", [(2, 2, 128, 30, 126, 70), (130, 1, 64, 20, 100, 60)])
def test_a_bad_page_that_one_row_sees_is_reported(nh, kvh, hs, past, q, pad):
    b, rules, unseen = _between_documents(nh, kvh, hs, past, q, pad)
    page = unseen[1]
    table = b.table.copy()
    table[0, page] = b.blocks
    b.meta = (*b.meta[:2], i32(table))
    rules.call(b)
    assert int(b.error) == 0
    j = (page + 1) * 16 - 1 - past  # the row of the page's last key sees that key alone
    rules.first[j] = past + j
    rules.call(b)
    assert int(b.error) == pa.DEVERR_BAD_BLOCK


# ---- values at the type's end ------------------------------------------------------------------


SATURATED = [([0], [40], {}, 0), ([300, 5], [70, 200], dict(softcap=20.0), 0),  # tiles
             ([3000], [12], {}, 0),                                             # a cluster's tile
             ([60], [3], {}, 4), ([60, 900, 0], [3, 4, 2], dict(bias=True), 0),  # rows: a cluster's, whole items, merged pieces
             ([9000] * 3, [4, 4, 1], {}, 4)]


@pytest.mark.parametrize("hs", [64, 128, 256])
@pytest.mark.parametrize("past,q,kw,longest", SATURATED)
def test_fp16_values_at_the_types_end_stay_finite(past, q, kw, longest, hs):
    """A mean of values of 65504 is 65504, however the weights are rounded on their way."""
    for seed in range(3):
        b = Batch(90 + seed, "fp16", 8, 2, hs, 16, past, q)
        for channel, value in ((3, 65504.0), (hs - 1, -65504.0)):
            v = b.value_cache[..., channel]
            v.copy_(torch.where(v.isnan(), v, torch.full_like(v, value)))
        rules = Rules(b, seed=3, bound=longest or None, **kw)
        out, lse = rules.call(b)
        assert int(b.error) == 0
        assert torch.isfinite(out).all()
        rules.check(b, out, lse)


@pytest.mark.parametrize("hs", [64, 128, 256])
@pytest.mark.parametrize("past,q,kw,longest", SATURATED)
def test_bf16_values_whose_sum_is_past_32_bits_keep_their_mean(past, q, kw, longest, hs):
    b = Batch(95, "bf16", 8, 2, hs, 16, past, q)
    v = b.value_cache[..., 5]
    top = torch.finfo(torch.bfloat16).max
    v.copy_(torch.where(v.isnan(), v, torch.full_like(v, top)))
    v = b.value_cache[..., 7]
    v.copy_(torch.where(v.isnan(), v, v.sign() * 2.0 ** 127))  # of both signs
    rules = Rules(b, seed=3, bound=longest or None, **kw)
    out, lse = rules.call(b)
    assert int(b.error) == 0
    assert torch.isfinite(out).all()
    rules.check(b, out, lse)


# ---- inputs rewritten right before the call ----------------------------------------------------


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nh,kvh,hs", [(8, 2, 128), (16, 2, 256), (32, 8, 64)])
def test_inputs_rewritten_right_before_a_mixed_call(nh, kvh, hs, dtype):
    """Prompts and decode rows in one call, whose kernels run side by side: each sees what the kernels right before the
    call have written to the query, the lengths, the table and the rules, and none of what stood there in the call before."""
    total = np.array([200, 300, 150, 400, 90, 700, 30, 600])
    qs = [[1, 40, 1, 90, 1, 2, 1, 1], [40, 1, 90, 1, 1, 1, 1, 2], [1, 1, 1, 1, 2, 60, 2, 69]]
    sets, want = [], []
    for seed, q in enumerate(qs):
        b = Batch(100 + seed, dtype, nh, kvh, hs, 16, total - q, q)
        rules = Rules(b, documents=200, prefix=40, bias=True, seed=seed)
        want.append(rules.call(b))
        assert int(b.error) == 0
        rules.check(b, *want[-1])
        sets.append([b.query.contiguous(), *b.meta, b.key_cache, b.value_cache, i32(rules.first), i32(rules.prefix),
                     torch.from_numpy(rules.slopes).cuda() * (1 + 0 * seed)])
    assert all(x.shape == y.shape for s in sets for x, y in zip(s, sets[0]))
    now = [t.clone() for t in sets[0]]

    def call(k):
        for t, x in zip(now, k):
            t.copy_(x)
        query, cum, past, table, kc, vc, first, prefix, slopes = now
        lse = torch.empty(query.shape[0], nh, device="cuda")
        out = pa.biased_paged_attention(query, kc, vc, cum, past, table, num_heads=nh, kv_num_heads=kvh, slopes=slopes,
                                        first_keys=first, prefix_lens=prefix, lse=lse)
        return out, lse

    for _ in range(4):
        got = [call(s) for s in sets]  # one after the other, nothing waited for
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    turn = [[t.clone() for t in s] for s in sets[:2]]  # what the graph's two calls are given
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        got = [call(s) for s in turn]
    for k in range(6):
        for i, s in enumerate(turn):
            for t, x in zip(s, sets[(k + i) % 3]):
                t.copy_(x)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            w = want[(k + i) % 3]
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


# ---- numbers that 32 bits cannot hold ------------------------------------------------------------


@pytest.mark.parametrize("fast", [True, False])
def test_a_cap_or_scale_that_32_bits_round_to_nothing_is_refused(fast, monkeypatch):
    """None of them may be taken for the 0 that stands for no cap, or for the scale by the head size."""
    if not fast:
        monkeypatch.setattr(pa.step, "_fast", _NoFast())
    b = Batch(110, "fp16", 8, 2, 64, 16, [40], [2])
    for kw in (dict(softcap=1e-60), dict(softcap=-1e-60), dict(scale=1e-60), dict(scale=-1e-60)):
        with pytest.raises(ValueError, match=next(iter(kw))):
            pa.biased_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, num_heads=8, kv_num_heads=2, **kw)
    pa.biased_paged_attention(b.query, b.key_cache, b.value_cache, *b.meta, num_heads=8, kv_num_heads=2, softcap=0, scale=0)


# ---- caps that are none ----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("softcap", [1e8, 1e30])
@pytest.mark.parametrize("hs,past,q,bound", [(128, [70, 0, 300], [1, 200, 150], 0), (256, [130, 20], [60, 1], 0), (64, [400], [2], 2),
                                             (128, [9000, 3], [1, 2], 2)])
def test_a_cap_far_above_all_scores_leaves_them(hs, past, q, bound, softcap, dtype):
    """Against the statement without a cap."""
    b = Batch(120, dtype, 8, 2, hs, 32, past, q)
    b.query[::2] *= 4
    for kw in (dict(), dict(bias=True, prefix=150)):
        rules, plain = (Rules(b, seed=9, softcap=c, bound=bound or None, **kw) for c in (softcap, 0.0))
        out, lse = rules.call(b)
        assert int(b.error) == 0
        o, z, size, mag, far = ref.biased_attention(
            f64(b.query).reshape(b.N, b.nh, hs), f64(b.key_cache), f64(b.value_cache), b.cum, b.past, b.table, hs ** -0.5,
            0.0, plain.slopes, 0, None, plain.prefix)
        # as Rules.check, but what the cap costs is in proportion to the score: the polynomial of three terms is 2^-19.4
        # off at a score of almost no size, the cap itself (s / c)^2 / 3, two products and the scale 2^-24 each
        delta = mag * ((hs + 8) * 2.0 ** -23 + 2.0 ** -19 + 2.0 ** -22) + far * 2.0 ** -22 + 2.0 ** -21 * (1 + np.abs(z))
        weight = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -16
        eps, tiny = torch.finfo(DT[dtype]).eps / 2, 2.0 ** -25 if dtype == "fp16" else 0.0
        bound_o = eps * np.abs(o) * (1 + 2.0 ** -7) + size * (weight + 2 * delta[..., None] + 2.0 ** -17) + tiny
        assert (np.abs(f64(out).reshape(o.shape) - o) <= bound_o).all()
        assert (np.abs(f64(lse) - z) <= delta + 2.0 ** -17).all()
        assert delta.max() < 0.05  # (so that a wrong score shows)


# ---- infinities and NaN that a row sees --------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("hs", [64, 128, 256])
@pytest.mark.parametrize("past,q,kw,longest", [
    ([200], [60], dict(), 0), ([0, 700], [300, 40], dict(bias=True), 0), ([3000], [12], dict(), 0),    # tiles, a cluster's
    ([0], [500], dict(documents=60, prefix=80), 0), ([100], [300], dict(window=90, softcap=20.0), 0),
    ([150], [3], dict(), 4), ([150, 900, 0], [3, 4, 2], dict(bias=True), 0), ([9000] * 3, [4, 4, 1], dict(softcap=9.0), 4)])
def test_values_that_a_row_sees_decide_its_channels_whatever_their_weights(past, q, kw, longest, hs, dtype):
    """An infinity is one and NaN is NaN in the rows that see it, however small its weight; infinities of both signs are
    NaN; all other rows and channels are as if it were not there."""
    b = Batch(130, dtype, 8, 2, hs, 16, past, q)
    rules = Rules(b, seed=4, bound=longest or None, **kw)
    plain = b.value_cache.clone()
    r = np.random.default_rng(5)
    for s in range(len(past)):
        total = past[s] + q[s]
        for channel, fills in ((1, [np.inf]), (2, [-np.inf]), (5, [np.nan]), (hs - 2, [np.inf, -np.inf]), (hs - 1, [np.inf, np.inf])):
            for fill in fills:
                t = int(r.integers(0, total)) if channel != 1 else int(r.integers(0, min(total, 20)))
                b.value_cache[b.table[s, t // 16], t % 16, 0, channel] = float(fill)
    out, lse = rules.call(b)
    assert int(b.error) == 0
    # what each row sees in each channel, from its range of keys
    want = np.zeros((b.N, 8, hs), int)  # 1: infinity, 2: minus infinity, 3: both, 4: NaN
    held = f64(b.value_cache)
    for s in range(len(past)):
        for j in range(q[s]):
            i = int(b.cum[s]) + j
            lo, hi = ref.key_range(past[s], q[s], j, rules.window, None if rules.first is None else int(rules.first[i]),
                                   None if rules.prefix is None else int(rules.prefix[s]))
            t = np.arange(lo, hi)
            v = held[b.table[s, t // 16], t % 16]  # (keys, kv heads, channels)
            for g in range(2):
                kind = np.isposinf(v[:, g]).any(0) * 1 | np.isneginf(v[:, g]).any(0) * 2 | np.isnan(v[:, g]).any(0) * 4
                want[i, g * 4: (g + 1) * 4] = kind
    got = f64(out).reshape(want.shape)
    assert (want == 0).any() and (want == 1).any()
    assert np.array_equal(np.isposinf(got), want == 1)
    assert np.array_equal(np.isneginf(got), want == 2)
    assert np.array_equal(np.isnan(got), want >= 3)
    clean = torch.where(torch.from_numpy(want != 0).cuda().flatten(1), torch.zeros_like(out), out)
    b.value_cache = plain
    o, z, size, mag, far = ref.biased_attention(
        f64(b.query).reshape(want.shape), f64(b.key_cache), f64(plain), b.cum, b.past, b.table, hs ** -0.5, rules.softcap,
        rules.slopes, rules.window, rules.first, rules.prefix)
    finite = np.where(np.isfinite(z), np.abs(z), 0)  # the bounds of Rules.check
    delta = mag * (hs + 8) * 2.0 ** -23 + far * 2.0 ** -22 + 2.0 ** -21 * (1 + finite + 2 * rules.softcap)
    weight = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -16
    eps, tiny = torch.finfo(DT[dtype]).eps / 2, 2.0 ** -25 if dtype == "fp16" else 0.0
    bound = eps * np.abs(o) * (1 + 2.0 ** -7) + size * (weight + 2 * delta[..., None] + 2.0 ** -17) + tiny
    assert (np.abs(f64(clean).reshape(want.shape) - o) <= bound)[want == 0].all()
    none = np.isneginf(z)
    assert np.array_equal(none, np.isneginf(f64(lse))) and (np.abs(f64(lse)[~none] - z[~none]) <= (delta + 2.0 ** -17)[~none]).all()


@pytest.mark.parametrize("past,q,longest", [([30], [3], 4), ([40, 900], [2, 2], 2), ([20], [60], 0)])
def test_an_infinite_value_of_no_weight_in_32_bits_is_infinite(past, q, longest):
    """A slope of 300 takes each key's weight to e^-300 of the next one's."""
    b = Batch(140, "bf16", 8, 2, 64, 16, past, q)
    rules = Rules(b, bias=True, bound=longest or None)
    rules.slopes[:] = 300.0
    for channel, fill in ((1, float("inf")), (40, float("-inf"))):
        b.value_cache[b.table[0, 0], 7, 1, channel] = fill
    out, lse = rules.call(b)
    got = f64(out).reshape(b.N, 8, 64)
    assert np.isposinf(got[: q[0], 4:, 1]).all() and np.isneginf(got[: q[0], 4:, 40]).all()
    got[: q[0], 4:, [1, 40]] = 0
    assert np.isfinite(got).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("past,q", [(50000, 1), (0, 4096)])
def test_what_a_value_that_is_not_finite_costs(past, q, dtype):
    """The header gives a row 0.05 ms for every 1000 keys; rows of a prompt share the chip's warps (over 900)."""
    b = Batch(141, dtype, 8, 2, 128, 16, [past], [q])
    rules = Rules(b, bound=q)
    b.value_cache[b.table[0, 0], 0, 0, 3] = float("inf")
    times = []
    for _ in range(4):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        out, _ = rules.call(b)
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end))
    assert torch.isposinf(out.view(-1, 8, 128)[:, :4, 3]).all()
    ms = 0.05 * (past + q) / 1000 if q == 1 else 0.05 * q / 2 / 1000 * (4 * q / 900)
    assert min(times) < 4 * ms + 1, (times, ms)
