"""The page operators and the biased attention, in their plain form and as the library's calls.

Four kinds of cases, each one pass through an operator as a serving loop calls it:

  fork     fork_block_tables: a new batch's rows from rows of the old one (beams that survive,
           samples of one prompt, requests that end), pages shared, copied on write or given back
  compact  compact_block_tables: the highest pages in use moved into the lowest free ones
  copy     copy_pages: the pages that either names, in the caches of all layers
  attend   biased_paged_attention: attention over the paged cache with capped scores, biases
           that grow with the distance, sliding windows, documents and prefixes

``own`` false computes them with elementary torch operations, true with the library.
"""
import math

import numpy as np
import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases -------------------------------------------------------------------------------


def listed():
    return [
        # a step of beam search: 16 prompts of 4 beams, some beams replaced by copies of others
        dict(name="fork: 16 prompts of 4 beams", op="fork", requests=64, group=4, keep=0.5, finished=0.0, longest=4096,
             block_size=64, pinned=0.0),
        # a busy server's step: samples of shared prompts, a tenth of the requests just ended
        dict(name="fork: 1024 requests", op="fork", requests=1024, group=8, keep=0.8, finished=0.1, longest=16384,
             block_size=16, pinned=0.02),
        # a small pool, mostly in order already
        dict(name="compact: 64 requests", op="compact", requests=64, longest=4096, block_size=64, fill=0.6, pinned=0.0,
             max_moves=64),
        # a large pool half empty, as many moves as it takes
        dict(name="compact: 1024 requests", op="compact", requests=1024, longest=8192, block_size=16, fill=0.5,
             pinned=0.02, max_moves=1 << 20),
        # the copies of a fork of few beams: one cache pair of one layer
        dict(name="copy: 24 pages of one layer", op="copy", entries=64, pages=24, layers=1, blocks=1024, block_size=64,
             kv_heads=8, head_size=128, dtype="fp16"),
        # a compaction's moves in the caches of all layers
        dict(name="copy: 160 pages of 24 layers", op="copy", entries=160, pages=160, layers=24, blocks=512,
             block_size=64, kv_heads=8, head_size=128, dtype="bf16"),
        # one request, one token: latency
        dict(name="attend: one decode row", op="attend", requests=1, past_lo=2047, past_hi=2047, rows=1, chunks=0,
             dtype="fp16", heads=32, kv_heads=8, head_size=128, block_size=64, softcap=50.0, bias=False, window=0,
             documents=0, prefix=0),
        # the decode batch of the dense benchmark's lengths with capped scores, 256-token pages
        dict(name="attend: 64 decode rows, cap", op="attend", requests=64, past_lo=512, past_hi=4096, rows=1, chunks=0,
             dtype="fp16", heads=32, kv_heads=8, head_size=128, block_size=256, softcap=50.0, bias=False, window=0,
             documents=0, prefix=0),
        # long histories in short pages, a bias by distance
        dict(name="attend: 8 long decode rows, bias", op="attend", requests=8, past_lo=32768, past_hi=131072, rows=1,
             chunks=0, dtype="bf16", heads=32, kv_heads=8, head_size=128, block_size=16, softcap=0.0, bias=True,
             window=0, documents=0, prefix=0),
        # drafted tokens of 256-wide heads, capped, in a window
        dict(name="attend: 32 requests of 5 drafts", op="attend", requests=32, past_lo=1024, past_hi=16384, rows=5,
             chunks=0, dtype="bf16", heads=16, kv_heads=2, head_size=256, block_size=32, softcap=30.0, bias=False,
             window=4096, documents=0, prefix=0),
        # chunked prompts beside decode rows, a sliding window
        dict(name="attend: 8 chunks, 24 decode, window", op="attend", requests=32, past_lo=1024, past_hi=16384,
             rows=512, chunks=8, dtype="fp16", heads=32, kv_heads=8, head_size=128, block_size=64, softcap=50.0,
             bias=False, window=4096, documents=0, prefix=0),
        # prompts with a bidirectional prefix, packed documents, a cap and a bias
        dict(name="attend: 4 prompts of 2048, all", op="attend", requests=4, past_lo=0, past_hi=8192, rows=2048,
             chunks=0, dtype="bf16", heads=32, kv_heads=8, head_size=128, block_size=256, softcap=50.0, bias=True,
             window=0, documents=6000, prefix=700),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fork", "compact", "copy", "attend", "attend", "attend"])
    heads, kv_heads, head_size = rng.choice([(32, 8, 128), (16, 2, 256), (16, 16, 64), (32, 4, 128), (14, 2, 64),
                                             (8, 1, 128)])
    if op == "fork":
        return dict(op=op, requests=_log(rng, 1, 1024), group=rng.randint(1, 8), keep=rng.choice([0.0, 0.5, 0.9]),
                    finished=rng.choice([0.0, 0.1, 0.5]), longest=_log(rng, 64, 16384),
                    block_size=rng.choice([16, 48, 64, 256]), pinned=rng.choice([0.0, 0.05]))
    if op == "compact":
        return dict(op=op, requests=_log(rng, 1, 1024), longest=_log(rng, 64, 8192),
                    block_size=rng.choice([16, 48, 64, 256]), fill=rng.uniform(0.2, 0.95),
                    pinned=rng.choice([0.0, 0.05]), max_moves=_log(rng, 1, 100000))
    if op == "copy":
        pages, layers = _log(rng, 1, 160), _log(rng, 1, 24)
        return dict(op=op, entries=pages + rng.choice([0, 1, 50]), pages=pages, layers=layers, blocks=2 * pages + rng.randint(0, 99),
                    block_size=rng.choice([16, 48, 64]), kv_heads=min(8, kv_heads), head_size=min(128, head_size),
                    dtype=rng.choice(["fp16", "bf16"]))
    kind = rng.choice(["decode", "drafts", "prompts"])
    if kind == "decode":
        past_hi = _log(rng, 64, 131072)
        requests, rows = _log(rng, 1, max(1, min(64, 524288 // past_hi))), 1
    elif kind == "drafts":
        past_hi = _log(rng, 256, 16384)
        rows, requests = rng.randint(2, 12), _log(rng, 1, max(1, min(32, 131072 // past_hi)))
    else:
        past_hi = _log(rng, 64, 8192)
        rows = _log(rng, 30, 2048)
        requests = rng.randint(1, max(1, 4096 // rows // 2))
    return dict(op=op, requests=requests, past_lo=rng.randint(0, past_hi), past_hi=past_hi, rows=rows,
                chunks=rng.choice([0, (requests + 1) // 2]), dtype=rng.choice(["fp16", "bf16"]), heads=heads,
                kv_heads=kv_heads, head_size=head_size, block_size=rng.choice([16, 32, 48, 64, 256]),
                softcap=rng.choice([0.0, 20.0, 50.0]), bias=rng.random() < 0.5,
                window=rng.choice([0, _log(rng, 1, 8192)]), documents=rng.choice([0, 0, _log(rng, 40, 8192)]),
                prefix=rng.choice([0, 0, _log(rng, 1, 1024)]))


# ---- lengths and pages: host arithmetic, from the seed alone ---------------------------------


def _lengths(case, seed):
    """(past, new rows) of every request of an attention case."""
    r = np.random.RandomState(seed % (1 << 32))
    n = case["requests"]
    past = r.randint(case["past_lo"], case["past_hi"] + 1, n)
    q = np.full(n, case["rows"])
    if case["chunks"]:  # the other requests have one row each
        q = np.where(r.permutation(n) < case["chunks"], q, 1)
    return past, q


def _masks(case, seed, past, q):
    """(first key of every row, prefix of every request): packed documents of about `documents`
    tokens, a few rows that are padding and see nothing; a prefix of up to `prefix` tokens."""
    r = np.random.RandomState((seed + 7) % (1 << 32))
    first, prefix = None, None
    if case["documents"]:
        first = []
        for b in range(len(past)):
            total = past[b] + q[b]
            ends = np.cumsum(r.randint(1, 2 * case["documents"], 2 + 3 * total // case["documents"]))
            p = past[b] + np.arange(q[b])
            starts = np.concatenate([[0], ends])[np.searchsorted(ends, p, side="right")]
            first.append(np.where(r.rand(q[b]) < 0.01, total, starts))
        first = np.concatenate(first)
    if case["prefix"]:
        prefix = r.randint(0, case["prefix"] + 1, len(past))
    return first, prefix


def _ranges(case, past, q, first, prefix):
    """The keys [lo, hi) of every row, and its request."""
    b = np.repeat(np.arange(len(q)), q)
    row = np.arange(len(b)) - np.repeat(np.cumsum(q) - q, q)
    p = past[b] + row
    lo = np.zeros_like(p) if first is None else first.copy()
    if case["window"]:
        lo = np.maximum(lo, p - case["window"] + 1)
    hi = p + 1 if prefix is None else np.maximum(p + 1, prefix[b])
    hi = np.minimum(hi, (past + q)[b])
    return lo, np.maximum(hi, lo), b


def _batch(case, seed):
    """A batch whose requests, in groups, share the whole pages of a common prompt: (lengths,
    pages held, table, the pool's pages that no request holds, its size)."""
    r = np.random.RandomState(seed % (1 << 32))
    n, bs = case["requests"], case["block_size"]
    group = case.get("group", 1)
    fixed = np.random.RandomState(n)  # the lengths are the case's, the groups' order the seed's
    past, more = fixed.randint(1, case["longest"] + 1, n), fixed.rand(n) < 0.1
    full = n // group * group
    turn = np.arange(full).reshape(-1, group)[r.permutation(full // group)].flatten()
    past[:full], more[:full] = past[turn], more[turn]
    common = np.repeat(np.minimum.reduceat(past, np.arange(0, n, group)) // 2 // bs, group)[:n]
    held = -(-past // bs) + more  # some still hold a page of refused drafts
    own_pages = held - common
    shared = common[::group]
    width = -(-case["longest"] // bs) + 2
    pages = int(own_pages.sum() + shared.sum())
    blocks = int(pages / case["fill"]) + 8 if "fill" in case else pages + n + 8
    order = r.permutation(blocks)
    table = np.full((n, width), -1)
    col = np.arange(width)
    first = np.cumsum(shared) - shared
    table = np.where(col < common[:, None], order[np.minimum(np.repeat(first, group)[:n, None] + col, blocks - 1)], table)
    start = shared.sum() + np.cumsum(own_pages) - own_pages
    at = start[:, None] + col - common[:, None]
    table = np.where((col >= common[:, None]) & (col < held[:, None]), order[np.clip(at, 0, blocks - 1)], table)
    return r, past, held, table, order[pages:], blocks


# ---- inputs ----------------------------------------------------------------------------------


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    return {"fork": _prepare_pages, "compact": _prepare_pages, "copy": _prepare_copy,
            "attend": _prepare_attend}[case["op"]](case, seed)


def _prepare_pages(case, seed):
    r, past, held, table, free, blocks = _batch(case, seed)
    n = len(past)
    s = {"case": case, "blocks": blocks, "past": _i32(past), "held": _i32(held), "table": _i32(table)}
    # some pages belong to a prefix cache as well, one of them to it alone
    pinned = r.rand(blocks) < case["pinned"]
    if case["pinned"] and len(free):
        pinned[free] = False
        pinned[free[-1]] = True
        free = free[:-1]
    s["pinned"] = torch.from_numpy(pinned).cuda() if case["pinned"] else None
    head = int(r.randint(0, blocks))
    ring = np.full(blocks, -1)
    ring[(head + np.arange(len(free))) % blocks] = free
    s["ring"], s["state"] = _i32(ring), _i32([head, len(free)])
    if case["op"] == "fork":
        group = case["group"]
        base = np.arange(n) // group * group
        other = base + r.randint(0, group, n) % np.maximum(np.minimum(group, n - base), 1)
        parents = np.where(r.rand(n) < case["keep"], np.arange(n), other)
        s["parents"] = _i32(np.where(r.rand(n) < case["finished"], -1, parents))
    return s


def _prepare_copy(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    shape = (case["blocks"], case["block_size"], case["kv_heads"], case["head_size"])
    order = r.permutation(case["blocks"])[: 2 * case["pages"]].reshape(-1, 2)
    copies = np.full((case["entries"], 2), -1)
    copies[: case["pages"]] = order
    caches = [torch.empty(shape, dtype=_DT[case["dtype"]], device="cuda").normal_(generator=gen)
              for _ in range(2 * case["layers"])]
    return {"case": case, "copies": _i32(copies), "caches": caches}


def _prepare_attend(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    past, q = _lengths(case, seed)
    nh, kvh, hs, bs, dt = case["heads"], case["kv_heads"], case["head_size"], case["block_size"], _DT[case["dtype"]]
    first, prefix = _masks(case, seed, past, q)
    total, n = past + q, int(q.sum())
    pages = -(-total // bs)
    width, blocks = -(-(case["past_hi"] + case["rows"]) // bs), int(pages.sum())
    order = torch.randperm(blocks, generator=gen, device="cuda").int()
    start = _i32(np.cumsum(pages) - pages)[:, None] + torch.arange(width, device="cuda", dtype=torch.int32)
    held = torch.arange(width, device="cuda") < _i32(pages)[:, None]
    s = {"case": case, "past": _i32(past), "cum": _i32(np.concatenate([[0], np.cumsum(q)])),
         "table": torch.where(held, order[start.clamp(max=blocks - 1).long()], -1)}
    s["key_cache"] = torch.empty(blocks, bs, kvh, hs, dtype=dt, device="cuda").normal_(generator=gen)
    s["value_cache"] = torch.empty(blocks, bs, kvh, hs, dtype=dt, device="cuda").normal_(generator=gen)
    s["query"] = (2 * rand(n, nh * hs)).to(dt)  # scores of a few units, as a trained model's
    s["first"] = None if first is None else _i32(first)
    s["prefix"] = None if prefix is None else _i32(prefix)
    # one rate per head, halving from head to head over eight octaves
    s["slopes"] = torch.exp2(-8 * torch.arange(1, nh + 1, device="cuda") / nh).float() if case["bias"] else None
    s["longest_rows"] = int(q.max())
    # the rows of the requests with several rows and of those with one, padded apart
    at = np.cumsum(q) - q
    many = q > 1
    rows = at[many][:, None] + np.arange(q.max())
    s["many"] = torch.from_numpy(np.where(np.arange(q.max()) < q[many][:, None], rows, -1)).cuda()
    s["ones"] = torch.from_numpy(at[q == 1][:, None]).cuda()
    s["of_many"], s["of_ones"] = (torch.from_numpy(np.flatnonzero(m)).cuda() for m in (many, q == 1))
    s["keys"] = [int(total[m].max()) if m.any() else 0 for m in (many, q == 1)]
    return s


# ---- one pass --------------------------------------------------------------------------------


def run(s):
    return {"fork": _run_fork, "compact": _run_compact, "copy": _run_copy, "attend": _run_attend}[s["case"]["op"]](s)


def _marks(pages, where, blocks):
    """Which pages of the pool are among `pages`."""
    marks = torch.zeros(blocks + 1, dtype=torch.bool, device=pages.device)
    return marks.index_fill(0, torch.where(where, pages, blocks).flatten().long(), True)[:blocks]


def _run_fork(s):
    bs, blocks = s["case"]["block_size"], s["blocks"]
    if own:
        import varlen_paged_kv_gb300 as pa
        t = pa.fork_block_tables(s["parents"], s["past"], s["held"], s["table"], s["ring"], s["state"], block_size=bs,
                                 num_blocks=blocks, pinned=s["pinned"])
        return [t.past_seqlens, t.blocks_held, t.block_table, t.copies, t.free_state, t.error, s["ring"]]
    parents, table, ring = s["parents"].long(), s["table"], s["ring"]
    dev, cap, width, n = table.device, ring.shape[0], table.shape[1], parents.shape[0]
    pinned = torch.zeros(blocks, dtype=torch.bool, device=dev) if s["pinned"] is None else s["pinned"]
    p = parents.clamp(min=0)
    past = torch.where(parents >= 0, s["past"][p].long(), 0)
    whole, need = past // bs, (past + bs - 1) // bs
    col, row = torch.arange(width, device=dev), torch.arange(n, device=dev)
    new = torch.where(col < need[:, None], table[p], -1).long()
    shared = _marks(new, col < whole[:, None], blocks)
    # the lowest row whose last page is partly filled keeps it, if nothing else holds it
    part = need > whole
    last = new.gather(1, whole.clamp(max=width - 1)[:, None])[:, 0]
    last = torch.where(part, last, blocks)
    keeper = torch.full((blocks + 1,), n, device=dev).scatter_reduce(0, last, row, "amin")
    taken = torch.cat([shared | pinned, shared.new_zeros(1)])[last]
    copy = part & (taken | (keeper[last] != row))
    rank = copy.long().cumsum(0) - copy.long()
    head, count = s["state"][0].long(), s["state"][1].long()
    to = ring[(head + rank) % cap].long()
    new = torch.where(copy[:, None] & (col == whole[:, None]), to[:, None], new)
    at = torch.where(copy, rank, n)
    copies = torch.full((n + 1, 2), -1, dtype=torch.int64, device=dev)
    copies = copies.index_copy(0, at, torch.stack([last, to], 1))[:n]
    # pages that were held and are not any more go behind the ring's last free page, in order
    gone = _marks(table, col < s["held"][:, None], blocks) & ~shared & (keeper[:blocks] == n) & ~pinned
    put = (head + count + gone.long().cumsum(0) - 1) % cap
    ring2 = torch.cat([ring, ring.new_zeros(1)]).index_copy(
        0, torch.where(gone, put, cap), torch.arange(blocks, device=dev, dtype=torch.int32))[:cap]
    took = copy.long().sum()
    state = torch.stack([(head + took) % cap, count - took + gone.long().sum()])
    i32 = torch.int32
    return [past.to(i32), need.to(i32), new.to(i32), copies.to(i32), state.to(i32),
            torch.zeros(1, dtype=i32, device=dev), ring2]


def _run_compact(s):
    blocks = s["blocks"]
    limit = min(s["case"]["max_moves"], blocks // 2)
    if own:
        import varlen_paged_kv_gb300 as pa
        t = pa.compact_block_tables(s["held"], s["table"], s["ring"], num_blocks=blocks, max_moves=limit,
                                    pinned=s["pinned"])
        return [t.block_table, t.copies, t.free_state, t.pages_end, t.error, s["ring"]]
    table, ring = s["table"], s["ring"]
    dev, i32 = table.device, torch.int32
    pinned = torch.zeros(blocks, dtype=torch.bool, device=dev) if s["pinned"] is None else s["pinned"]
    held = torch.arange(table.shape[1], device=dev) < s["held"][:, None]
    used = _marks(table, held, blocks) | pinned
    page = torch.arange(blocks, device=dev)
    mover, hole = (used & ~pinned).long(), (~used).long()
    below = hole.cumsum(0) - hole                                # holes below a page
    above = mover.sum() - mover.cumsum(0)                        # movers above it
    holes = torch.zeros(blocks + 1, dtype=torch.int64, device=dev)
    holes = holes.index_copy(0, torch.where(hole > 0, below, blocks), page)
    moves = (mover > 0) & (above < limit) & (below > above)
    to = torch.where(moves, holes[above], page)
    new = torch.where(held, to[table.clamp(min=0).long()].to(i32), table)
    copies = torch.full((limit + 1, 2), -1, dtype=torch.int64, device=dev)
    copies = copies.index_copy(0, torch.where(moves, above, limit), torch.stack([page, to], 1))[:limit]
    after = _marks(to, used, blocks)
    free = (~after).long()
    ring2 = torch.cat([ring, ring.new_zeros(1)]).index_copy(
        0, torch.where(after, ring.shape[0], free.cumsum(0) - free), page.to(i32))[: ring.shape[0]]
    state = torch.stack([free.sum() * 0, free.sum()])
    end = torch.where(after, page + 1, 0).amax()[None]
    return [new, copies.to(i32), state.to(i32), end.to(i32), torch.zeros(1, dtype=i32, device=dev), ring2]


def _run_copy(s):
    if own:
        import varlen_paged_kv_gb300 as pa
        pa.copy_pages(s["caches"], s["copies"])
        return s["caches"]
    src, dst = s["copies"][:, 0].long(), s["copies"][:, 1].long()
    some = src >= 0
    any_one = some.long().argmax()  # an entry of -1 makes one of the copies once more
    src, dst = torch.where(some, src, src[any_one]), torch.where(some, dst, dst[any_one])
    return [c.index_copy_(0, dst, c[src]) for c in s["caches"]]


def _plain_rows(s, rows, request, keys):
    """(out, lse) of padded rows (requests, rows) over the first `keys` keys of their requests."""
    c = s["case"]
    nh, kvh, hs, bs = (c[k] for k in ("heads", "kv_heads", "head_size", "block_size"))
    G, at = nh // kvh, rows.clamp(min=0)
    width = (keys + bs - 1) // bs
    page = s["table"][request, :width].clamp(min=0).long()
    k, v = (s[x][page].flatten(1, 2).permute(0, 2, 3, 1).float() for x in ("key_cache", "value_cache"))
    q = s["query"].unflatten(1, (kvh, G, hs))[at].float()                 # (b, r, kvh, G, hs)
    w = torch.matmul(q.permute(0, 2, 3, 1, 4).flatten(2, 3), k)           # (b, kvh, G r, keys)
    w = w.unflatten(2, (G, rows.shape[1])).mul_(1 / math.sqrt(hs))
    if c["softcap"]:
        w = w.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    past, cum = s["past"][request], s["cum"][request]
    total = past + s["cum"][request + 1] - cum
    pos = past[:, None] + at - cum[:, None]                               # (b, r)
    key = torch.arange(k.shape[3], device=w.device)
    if c["bias"]:
        far = (pos[..., None] - key).abs().float()
        w = w.sub_(s["slopes"].reshape(kvh, G)[:, :, None, None] * far[:, None, None])
    lo = torch.zeros_like(pos) if s["first"] is None else s["first"][at]
    if c["window"]:
        lo = torch.maximum(lo, pos - (c["window"] - 1))
    hi = pos + 1 if s["prefix"] is None else torch.maximum(pos + 1, s["prefix"][request][:, None])
    hi = torch.minimum(hi, total[:, None])
    seen = (key >= lo[..., None]) & (key < hi[..., None])
    w = w.masked_fill_(~seen[:, None, None], -math.inf)
    most = w.amax(4, keepdim=True)
    w = w.sub_(torch.where(most == -math.inf, 0.0, most)).exp_()
    sums = w.sum(4, keepdim=True)
    o = torch.matmul(w.flatten(2, 3), v.transpose(2, 3)).unflatten(2, (G, rows.shape[1]))
    o = torch.where(sums > 0, o / sums, 0.0).permute(0, 3, 1, 2, 4).flatten(2)
    lse = (most + torch.log(sums))[..., 0].permute(0, 3, 1, 2).flatten(2)
    return o, lse


def _run_attend(s):
    c = s["case"]
    n, nh = s["query"].shape[0], c["heads"]
    if own:
        import varlen_paged_kv_gb300 as pa
        lse = torch.empty(n, nh, dtype=torch.float32, device="cuda")
        out = pa.biased_paged_attention(
            s["query"], s["key_cache"], s["value_cache"], s["cum"], s["past"], s["table"], num_heads=nh,
            kv_num_heads=c["kv_heads"], softcap=c["softcap"], slopes=s["slopes"], window=c["window"],
            first_keys=s["first"], prefix_lens=s["prefix"], max_query_len=s["longest_rows"], lse=lse)
        return [out, lse]
    out, lse = s["query"].new_empty(n + 1, s["query"].shape[1]), torch.empty(n + 1, nh, device="cuda")

    def group(out, lse, rows, request, keys):
        if not keys:
            return out, lse
        o, z = _plain_rows(s, rows, request, keys)
        to = torch.where(rows >= 0, rows, n).flatten()
        return out.index_copy_(0, to, o.flatten(0, 1).to(out.dtype)), lse.index_copy_(0, to, z.flatten(0, 1))

    out, lse = group(out, lse, s["many"], s["of_many"], s["keys"][0])
    out, lse = group(out, lse, s["ones"], s["of_ones"], s["keys"][1])
    return [out[:n], lse[:n]]


# ---- what a pass cannot do without -----------------------------------------------------------


def work(case):
    if case["op"] == "copy":
        page = case["block_size"] * case["kv_heads"] * case["head_size"] * 2
        return {"bytes": 2 * 2 * case["layers"] * case["pages"] * page + 8 * case["entries"], "flops": 0}
    if case["op"] != "attend":
        _, _, held, table, _, blocks = _batch(case, 0)
        entries = int(held.sum()) + table.size  # the held pages read, the new table written
        if case["op"] == "compact":
            entries += 2 * min(case["max_moves"], blocks // 2) + blocks - int(held.sum())
        else:
            entries += 10 * len(held)
        return {"bytes": 4 * entries, "flops": 2 * entries}
    past, q = _lengths(case, 0)
    lo, hi, b = _ranges(case, past, q, *_masks(case, 0, past, q))
    nh, kvh, hs = case["heads"], case["kv_heads"], case["head_size"]
    some = hi > lo
    low, high = np.full(len(q), 1 << 40), np.zeros(len(q), np.int64)
    np.minimum.at(low, b[some], lo[some])
    np.maximum.at(high, b[some], hi[some])
    keys = int(np.maximum(high - low, 0).sum())
    return {"bytes": keys * kvh * hs * 4 + len(b) * nh * (4 * hs + 4) + 4 * keys // case["block_size"],
            "flops": int((hi - lo).sum()) * nh * hs * 4}


# ---- the definitions in 64 bits --------------------------------------------------------------


def exact(case, seed):
    if case["op"] != "attend":
        return None  # whole numbers and copies only
    s = _prepare_attend(case, seed)
    past, q = _lengths(case, seed)
    lo, hi, _ = _ranges(case, past, q, *_masks(case, seed, past, q))
    nh, kvh, hs, bs = (case[k] for k in ("heads", "kv_heads", "head_size", "block_size"))
    G, cum = nh // kvh, np.concatenate([[0], np.cumsum(q)])
    out = torch.zeros(cum[-1], nh, hs, dtype=torch.float64, device="cuda")
    lse = torch.full((cum[-1], nh), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(len(q)):
        page = s["table"][b, : -(-(past[b] + q[b]) // bs)].long()
        keys, values = s["key_cache"][page].flatten(0, 1), s["value_cache"][page].flatten(0, 1)
        step = max(1, (1 << 27) // (G * (past[b] + q[b])))
        for r0 in range(cum[b], cum[b + 1], step):
            r1 = min(cum[b + 1], r0 + step)
            k0, k1 = int(lo[r0:r1].min()), int(hi[r0:r1].max())
            k1 = min(k1, past[b] + q[b])
            if k1 <= k0:
                continue
            j = torch.arange(k0, k1, device="cuda")
            begin, end = (torch.from_numpy(x[r0:r1]).cuda()[:, None] for x in (lo, hi))
            seen = (begin <= j) & (j < end)                               # (rows, keys)
            away = (past[b] + torch.arange(r0, r1, device="cuda") - cum[b])[:, None] - j
            for g in range(kvh):
                rows = s["query"][r0:r1].reshape(r1 - r0, nh, hs)[:, g * G: (g + 1) * G].double()
                z = rows.transpose(0, 1) @ keys[k0:k1, g].double().T / hs ** 0.5     # (G, rows, keys)
                if case["softcap"]:
                    z = torch.tanh(z / case["softcap"]) * case["softcap"]
                if case["bias"]:
                    z -= s["slopes"][g * G: (g + 1) * G].double()[:, None, None] * away.abs().double()
                z.masked_fill_(~seen, -math.inf)
                total = torch.logsumexp(z, 2)
                z = torch.exp(z - torch.where(total == -math.inf, 0.0, total)[..., None])
                out[r0:r1, g * G: (g + 1) * G] = (z @ values[k0:k1, g].double()).transpose(0, 1)
                lse[r0:r1, g * G: (g + 1) * G] = total.T
    return [out.flatten(1), lse]
