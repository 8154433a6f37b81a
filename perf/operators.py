"""The operators around paged attention, in their plain form and as the library's calls.

Four kinds of cases, each one pass through an operator as a serving loop calls it:

  tables  build_block_tables: the step's prefix sums, positions, slots and block tables from
          the requests' lengths, pages taken from and returned to a ring of free pages
  rotate  qk_norm_rope: RMSNorm of every query and key head, then the rotary embedding
  bounds  update_page_bounds: the per-page minimum and maximum codes of the keys just cached
  sparse  select_pages, then sparse_paged_attention over the selected pages

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
        # a decode step: every request has one new token, some cross into a new page
        dict(name="tables: 64 requests decoding", op="tables", requests=64, decoding=1.0, chunk=1, finished=0.0,
             longest=4096, block_size=256),
        # a busy server's step: chunked prompts beside decoding requests, some just finished
        dict(name="tables: 1024 requests, chunks of 512", op="tables", requests=1024, decoding=0.9, chunk=512,
             finished=0.05, longest=16384, block_size=16),
        # one decode batch, packed [Q | K | V] rows
        dict(name="rotate: 64 decode rows", op="rotate", tokens=64, dtype="fp16", heads=32, kv_heads=8, head_size=128,
             rotary=128, interleaved=False, norm=True, packed=True),
        # a prompt chunk of 256-wide heads with a quarter of each rotated, an odd number of rows
        dict(name="rotate: 8001 prompt rows, wide heads", op="rotate", tokens=8001, dtype="bf16", heads=16, kv_heads=2,
             head_size=256, rotary=64, interleaved=False, norm=True, packed=False),
        # one new key per request
        dict(name="bounds: 64 decode rows", op="bounds", requests=64, past_lo=512, past_hi=4096, rows=1, dtype="fp16",
             kv_heads=8, head_size=128, block_size=64),
        # prompts just written to the cache, starting inside a page
        dict(name="bounds: 4 prompts of 2048", op="bounds", requests=4, past_lo=0, past_hi=8192, rows=2048,
             dtype="bf16", kv_heads=8, head_size=128, block_size=64),
        # one request with a long history: latency
        dict(name="sparse: one long request", op="sparse", requests=1, past_lo=131071, past_hi=131071, rows=1,
             chunks=0, dtype="fp16", heads=32, kv_heads=8, head_size=128, block_size=64, top_k=32, query_block=1),
        # the decode batch of the dense benchmark, a quarter to all of each history selected
        dict(name="sparse: 64 decode rows", op="sparse", requests=64, past_lo=512, past_hi=4096, rows=1, chunks=0,
             dtype="fp16", heads=32, kv_heads=8, head_size=128, block_size=64, top_k=16, query_block=1),
        # long histories in short pages
        dict(name="sparse: 8 long decode rows", op="sparse", requests=8, past_lo=32768, past_hi=131072, rows=1,
             chunks=0, dtype="bf16", heads=32, kv_heads=8, head_size=128, block_size=16, top_k=128, query_block=1),
        # drafted tokens: four rows of a request share one selection, 256-wide heads
        dict(name="sparse: 32 requests of 4 drafts", op="sparse", requests=32, past_lo=4096, past_hi=32768, rows=4,
             chunks=0, dtype="fp16", heads=16, kv_heads=2, head_size=256, block_size=32, top_k=48, query_block=4),
        # chunked prompts beside decode rows, blocks of 16 queries
        dict(name="sparse: 8 chunks of 512, 24 decode", op="sparse", requests=32, past_lo=1024, past_hi=16384, rows=512,
             chunks=8, dtype="fp16", heads=32, kv_heads=8, head_size=128, block_size=64, top_k=32, query_block=16),
        # long prompts in blocks of 32 queries
        dict(name="sparse: 4 prompts of 2048", op="sparse", requests=4, past_lo=8192, past_hi=32768, rows=2048,
             chunks=0, dtype="bf16", heads=32, kv_heads=8, head_size=128, block_size=64, top_k=32, query_block=32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rotate", "bounds", "sparse", "sparse", "sparse"])
    dtype = rng.choice(["fp16", "bf16"])
    heads, kv_heads, head_size = rng.choice([(32, 8, 128), (16, 2, 256), (16, 16, 64), (32, 4, 128), (14, 2, 64),
                                             (8, 1, 128)])
    if op == "tables":
        return dict(op=op, requests=_log(rng, 1, 1024), decoding=rng.choice([1.0, 0.9, 0.5]), chunk=_log(rng, 2, 512),
                    finished=rng.choice([0.0, 0.05, 0.3]), longest=_log(rng, 512, 16384),
                    block_size=rng.choice([16, 48, 64, 256]))
    if op == "rotate":
        return dict(op=op, tokens=_log(rng, 1, 8001), dtype=dtype, heads=heads, kv_heads=kv_heads,
                    head_size=head_size, rotary=rng.choice([head_size, head_size // 2, head_size // 4, 0]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7, packed=rng.random() < 0.5)
    if op == "bounds":
        rows = _log(rng, 1, 2048)
        return dict(op=op, requests=_log(rng, 1, max(1, min(64, 8192 // rows))), past_lo=0, past_hi=_log(rng, 1, 8192),
                    rows=rows, dtype=dtype, kv_heads=kv_heads, head_size=head_size,
                    block_size=rng.choice([16, 32, 48, 64, 256]))
    block_size = rng.choice([16, 32, 48, 64, 128])
    kind = rng.choice(["decode", "drafts", "prompts"])
    if kind == "decode":
        past_hi = _log(rng, 64, 131072)
        requests, rows, query_block = _log(rng, 1, max(1, min(64, 524288 // past_hi))), 1, 1
    elif kind == "drafts":
        past_hi = _log(rng, 256, 32768)
        rows = rng.randint(2, 8)
        requests, query_block = _log(rng, 1, max(1, min(32, 262144 // past_hi))), rng.choice([1, rows])
    else:
        past_hi = _log(rng, 64, 16384)
        rows = _log(rng, 100, 2048)
        requests, query_block = rng.randint(1, max(1, 4096 // rows)), rng.choice([16, 32, 64])
    top_k = _log(rng, 4, max(5, 2048 // block_size)) + (query_block + block_size - 2) // block_size
    return dict(op=op, requests=requests, past_lo=rng.randint(0, past_hi), past_hi=past_hi, rows=rows,
                chunks=rng.choice([0, (requests + 1) // 2]), dtype=dtype, heads=heads, kv_heads=kv_heads,
                head_size=head_size, block_size=block_size, top_k=top_k, query_block=query_block)


# ---- lengths: host arithmetic, from the seed alone -------------------------------------------


def _lengths(case, seed):
    """(past, new rows) of every request."""
    r = np.random.RandomState(seed % (1 << 32))
    n = case["requests"]
    fixed = np.random.RandomState(n)  # the step's row counts are the case's, their order the seed's
    if case["op"] == "tables":
        ends, ones = int(n * case["finished"]), int(n * case["decoding"])
        q = fixed.randint(1, case["chunk"] + 1, n)
        q[:ones] = 1
        q[:ends] = -1
        return r.randint(0, case["longest"], n), r.permutation(q)
    past = r.randint(case["past_lo"], case["past_hi"] + 1, n)
    q = np.full(n, case["rows"])
    if case["op"] == "bounds":  # half of the requests have fewer rows
        q[n // 2 + 1:] = fixed.randint(1, case["rows"] + 1, n - n // 2 - 1)
        q = r.permutation(q)
    if case["op"] == "sparse" and case["chunks"]:  # the other requests have one row each
        q = np.where(r.permutation(n) < case["chunks"], q, 1)
    return past, q


def _cum(q):
    return np.concatenate([[0], np.cumsum(np.maximum(q, 0))])


def _blocks(case, q):
    """Rows of every query block, (blocks, query_block), and the request of each; -1 past its end."""
    R, cum = case["query_block"], _cum(q)
    rows, request = [], []
    for b in range(len(q)):
        first = np.arange(cum[b], cum[b + 1], R)
        at = first[:, None] + np.arange(R)
        rows.append(np.where(at < cum[b + 1], at, -1))
        request.append(np.full(len(first), b))
    return np.concatenate(rows), np.concatenate(request)


# ---- inputs ----------------------------------------------------------------------------------


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _table(pages, blocks, width, gen):
    """A block table whose requests hold `pages` pages each of a pool of `blocks`, and the pool's order."""
    order = torch.randperm(blocks, generator=gen, device="cuda").int()
    start = np.concatenate([[0], np.cumsum(pages)])
    at = _i32(start[:-1])[:, None] + torch.arange(width, device="cuda", dtype=torch.int32)
    held = torch.arange(width, device="cuda") < _i32(pages)[:, None]
    return torch.where(held, order[at.clamp(max=max(blocks - 1, 0)).long()], -1), order


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "rotate":
        n, nh, kvh, hs = case["tokens"], case["heads"], case["kv_heads"], case["head_size"]
        dt = _DT[case["dtype"]]
        row = rand(n, (nh + 2 * kvh) * hs).to(dt)
        if case["packed"]:  # views of packed [Q | K | V] rows
            s["query"], s["key"] = row[:, : nh * hs], row[:, nh * hs: (nh + kvh) * hs]
        else:
            s["query"], s["key"] = row[:, : nh * hs].contiguous(), row[:, nh * hs: (nh + kvh) * hs].contiguous()
        s["positions"] = torch.randint(0, 131072, (n,), generator=gen, device="cuda", dtype=torch.int32)
        norm = case["norm"]
        s["q_weight"] = (1 + 0.2 * rand(hs)).to(dt) if norm else None
        s["k_weight"] = (1 + 0.2 * rand(hs)).to(dt) if norm else None
        return s
    past, q = _lengths(case, seed)
    bs = case["block_size"]
    s["past"], s["num_tokens"] = _i32(past), int(_cum(q)[-1])
    if case["op"] == "tables":
        r = np.random.RandomState((seed + 1) % (1 << 32))
        held = -(-past // bs) + (r.rand(len(q)) < 0.1)  # some still hold a page of refused drafts
        need = np.where(q > 0, -(-(past + np.maximum(q, 0)) // bs), 0)
        width = -(-(case["longest"] + case["chunk"]) // bs) + 1
        blocks = len(q) * width  # every request could grow to the longest
        s["block_table"], order = _table(held, blocks, width, gen)
        free = blocks - int(held.sum())  # the pages that no request holds, from a place of the ring on
        head = int(r.randint(0, blocks))
        ring = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
        ring[(head + torch.arange(free, device="cuda")) % blocks] = order[int(held.sum()):]
        s["free_blocks"] = ring
        s["num_tokens"] = -(-s["num_tokens"] // 64) * 64  # a captured step's row count: the rows behind are no one's
        s["query_lens"], s["held"], s["free_state"] = _i32(q), _i32(held), _i32([head, free])
        return s
    kvh, hs, dt = case["kv_heads"], case["head_size"], _DT[case["dtype"]]
    pages = -(-(past + q) // bs)
    longest = -(-(case["past_hi"] + case["rows"]) // bs)
    blocks = len(q) * longest if case["op"] == "bounds" else int(pages.sum())
    s["block_table"], _ = _table(pages, blocks, longest, gen)
    s["cum"] = _i32(_cum(q))
    # keys of a page share a direction (neighbouring tokens are alike), a few channels are large
    centre = 0.8 * rand(blocks, 1, kvh, hs)
    gain = 1 + 2 * (torch.rand(kvh, hs, generator=gen, device="cuda") < 0.04)
    s["key_cache"] = torch.empty(blocks, bs, kvh, hs, dtype=dt, device="cuda")
    for at in range(0, blocks, 4096):  # in pieces: the 32-bit values of a whole cache need not be held
        c = centre[at: at + 4096]
        s["key_cache"][at: at + 4096] = ((c + 0.6 * rand(c.shape[0], bs, kvh, hs)) * gain).to(dt)
    s["scale"] = (gain * 3.5 / 127).float().contiguous()
    code = lambda x: (x.float() / s["scale"]).round().clamp(-127, 127).to(torch.int8)  # noqa: E731
    if case["op"] == "bounds":
        # before the call the bounds cover the keys that were there already
        lo, hi = code(s["key_cache"][:, :1].amin(1)), code(s["key_cache"][:, :1].amax(1))
        s["bounds"] = torch.stack([lo, hi], 2).contiguous()
        return s
    nh = case["heads"]
    s["bounds"] = torch.stack([code(s["key_cache"].amin(1)), code(s["key_cache"].amax(1))], 2).contiguous()
    s["value_cache"] = torch.empty_like(s["key_cache"])
    for at in range(0, blocks, 4096):
        v = s["value_cache"][at: at + 4096]
        v.copy_(rand(*v.shape))
    rows, request = _blocks(case, q)
    s["rows"] = torch.from_numpy(rows).cuda()
    s["request"] = torch.from_numpy(request).cuda()
    # a query looks for a few pages of its request: a block's queries for the same ones
    n, G = s["num_tokens"], nh // kvh
    want = torch.rand(len(rows), 3, generator=gen, device="cuda") * _i32(pages)[s["request"]][:, None]
    page = s["block_table"][s["request"][:, None], want.long()].long()
    target = centre[page, 0].sum(1)                                    # (blocks of queries, kvh, hs)
    of_row = torch.zeros(n, dtype=torch.long, device="cuda")
    of_row[s["rows"].clamp(min=0).flatten()] = torch.arange(len(rows), device="cuda").repeat_interleave(rows.shape[1])
    query = torch.empty(n, nh * hs, dtype=dt, device="cuda")
    first = s["rows"][:, 0]
    start = torch.searchsorted(first, torch.arange(n, device="cuda"), right=True) - 1
    for at in range(0, n, 2048):
        t = target[start[at: at + 2048]].unsqueeze(2)
        query[at: at + 2048] = ((0.5 * t + rand(t.shape[0], kvh, G, hs)) / gain[:, None]).to(dt).flatten(1)
    s["query"] = query
    return s


# ---- one pass --------------------------------------------------------------------------------


def run(s):
    return {"tables": _run_tables, "rotate": _run_rotate, "bounds": _run_bounds, "sparse": _run_sparse}[s["case"]["op"]](s)


def _run_tables(s):
    bs, n = s["case"]["block_size"], s["num_tokens"]
    if own:
        import varlen_paged_kv_gb300 as pa
        t = pa.build_block_tables(s["past"], s["query_lens"], s["held"], s["block_table"], s["free_blocks"],
                                  s["free_state"], block_size=bs, num_tokens=n)
        return [t.cumulative_sequence_length, t.slot_mapping, t.positions, t.blocks_held, t.free_state, t.error,
                s["block_table"], s["free_blocks"]]
    past, held, table, ring = s["past"].long(), s["held"].long(), s["block_table"], s["free_blocks"]
    B, width = table.shape
    cap = ring.shape[0]
    q = s["query_lens"].long().clamp(min=0)
    gone = s["query_lens"] < 0
    need = torch.where(q > 0, (past + q + bs - 1) // bs, 0)
    grow = (need - held).clamp(min=0)
    back = torch.where(gone, held, 0)
    cum = torch.cat([q.new_zeros(1), q.cumsum(0)])
    head, count = s["free_state"][0].long(), s["free_state"][1].long()
    col = torch.arange(width, device=table.device)
    took = grow.cumsum(0) - grow
    at = (head + took[:, None] + col - held[:, None]) % cap
    new = (col >= held[:, None]) & (col < need[:, None])
    table2 = torch.where(new, ring[at], table)
    # the finished requests' pages go behind the ring's last free page, in request order
    put = (head + count + (back.cumsum(0) - back)[:, None] + col) % cap
    put = torch.where(col < back[:, None], put, cap)
    ring2 = torch.cat([ring, ring.new_zeros(1)]).scatter(0, put.flatten(), table.flatten())[:cap]
    token = torch.arange(n, device=table.device)
    b = torch.searchsorted(cum[1:], token, right=True).clamp(max=B - 1)
    there = token < cum[-1]
    pos = torch.where(there, past[b] + token - cum[b], -1)
    at = torch.where(there, pos, 0)
    slot = torch.where(there, table2[b, at // bs] * bs + at % bs, -1)
    state = torch.stack([(head + grow.sum()) % cap, count - grow.sum() + back.sum()])
    left = torch.where(gone, 0, held + grow)
    i32 = torch.int32
    return [cum.to(i32), slot.to(i32), pos.to(i32), left.to(i32), state.to(i32),
            torch.zeros(1, dtype=i32, device=table.device), table2, ring2]


def _run_rotate(s):
    c = s["case"]
    nh, kvh, hs, d = c["heads"], c["kv_heads"], c["head_size"], c["rotary"]
    if own:
        import varlen_paged_kv_gb300 as pa
        return list(pa.qk_norm_rope(s["query"], s["key"], s["positions"], num_heads=nh, kv_num_heads=kvh,
                                    q_norm_weight=s["q_weight"], k_norm_weight=s["k_weight"], eps=1e-6, rotary_dim=d,
                                    theta=1e6, interleaved=c["interleaved"]))
    if d:
        # a 32-bit table of the frequencies and the 32-bit product with the position define the angle
        freq = torch.pow(1e6, -2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d).float()
        angle = (s["positions"].float()[:, None] * freq).double()
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, heads, w):
        x = x.unflatten(1, (heads, hs)).float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(2, keepdim=True) + 1e-6) * w.float()
        if d:
            if c["interleaved"]:
                u, v = x[..., 0:d:2], x[..., 1:d:2]
                turned = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(2)
            else:
                u, v = x[..., : d // 2], x[..., d // 2: d]
                turned = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
            x = torch.cat([turned, x[..., d:]], -1)
        return x.flatten(1).to(_DT[c["dtype"]])

    return [one(s["query"], nh, s["q_weight"]), one(s["key"], kvh, s["k_weight"])]


def _run_bounds(s):
    bs, n = s["case"]["block_size"], s["num_tokens"]
    if own:
        import varlen_paged_kv_gb300 as pa
        return pa.update_page_bounds(s["key_cache"], s["bounds"], s["scale"], s["cum"], s["past"], s["block_table"],
                                     num_tokens=n)
    # every new key's code into its page; a page that the call begins starts afresh
    token = torch.arange(n, device="cuda")
    b = torch.searchsorted(s["cum"][1:], token.int(), right=True)
    pos = s["past"][b] + token - s["cum"][b]
    page = s["block_table"][b, pos // bs].long()
    code = (s["key_cache"][page, pos % bs].float() / s["scale"]).round().clamp(-127, 127).to(torch.int8)
    blocks = s["bounds"].shape[0]
    fresh = torch.zeros(blocks + 1, dtype=torch.bool, device="cuda")
    fresh = fresh.index_fill(0, torch.where(pos % bs == 0, page, blocks), True)[:-1, None, None]
    lo = torch.where(fresh, 127, s["bounds"][:, :, 0])
    hi = torch.where(fresh, -127, s["bounds"][:, :, 1])
    at = page[:, None, None].expand_as(code)
    lo = lo.to(torch.int8).scatter_reduce(0, at, code, "amin")
    hi = hi.to(torch.int8).scatter_reduce(0, at, code, "amax")
    return torch.stack([lo, hi], 2)


def _run_sparse(s):
    c = s["case"]
    nh, kvh, hs, bs, K, R = (c[k] for k in ("heads", "kv_heads", "head_size", "block_size", "top_k", "query_block"))
    n = s["num_tokens"]
    if own:
        import varlen_paged_kv_gb300 as pa
        sel = pa.select_pages(s["query"], s["bounds"], s["scale"], s["cum"], s["past"], s["block_table"], num_heads=nh,
                              kv_num_heads=kvh, block_size=bs, top_k=K, query_block=R)
        lse = torch.empty(n, nh, dtype=torch.float32, device="cuda")
        out = pa.sparse_paged_attention(s["query"], s["key_cache"], s["value_cache"], s["cum"], s["past"],
                                        s["block_table"], sel, num_heads=nh, kv_num_heads=kvh, query_block=R, lse=lse)
        return [sel, out, lse]
    G, rows, b = nh // kvh, s["rows"], s["request"]
    there = rows >= 0                                                         # (blocks, R)
    at = rows.clamp(min=0)
    q = s["query"].unflatten(1, (kvh, G, hs))[at].float()                     # (blocks, R, kvh, G, hs)
    pos = torch.where(there, s["past"][b][:, None] + at - s["cum"][b][:, None], -1)
    # the block's codes: 12-bit codes of every row, summed by sign, rescaled to 8 bits
    x = q * s["scale"][:, None] * there[:, :, None, None, None]
    most = x.abs().amax((1, 3, 4), keepdim=True)
    fine = torch.full_like(most, 4095) / most  # one rounding (a scalar over a tensor takes two)
    code = (x * torch.where(most > 1e-30, fine, 0.0)).round().long()
    plus, minus = code.clamp(min=0).sum((1, 3)), (-code).clamp(min=0).sum((1, 3))      # (blocks, kvh, hs)
    m = torch.maximum(plus, minus).amax(2, keepdim=True).clamp(min=1)
    plus, minus = ((510 * plus + m) // (2 * m)).float(), ((510 * minus + m) // (2 * m)).float()
    # scores of all pages of the request (whole numbers below 2^24, so exact in 32 bits)
    pages = s["block_table"].shape[1]
    bound = s["bounds"][s["block_table"][b].clamp(min=0).long()].float()     # (blocks, pages, kvh, 2, hs)
    score = torch.einsum("nkd,npkd->nkp", plus, bound[:, :, :, 1]) - torch.einsum("nkd,npkd->nkp", minus, bound[:, :, :, 0])
    del bound
    page = torch.arange(pages, device="cuda")
    first, last = (pos[:, 0] // bs)[:, None, None], (pos.amax(1) // bs)[:, None, None]
    score = torch.where((page < 1) | (page >= first), 1e9, score)             # the first page, and the rows' own
    score = torch.where(page > last, -1e9, score)
    best = torch.sort(score, dim=2, descending=True, stable=True)
    best = best.indices[..., :K] if K <= pages else torch.nn.functional.pad(best.indices, (0, K - pages), value=pages)
    best = torch.where(best > last, 1 << 30, best).sort(2).values
    some = best < (1 << 30)
    # attention of the block's rows over the selected pages
    phys = s["block_table"][b[:, None, None], torch.where(some, best, 0)].long()      # (blocks, kvh, K)
    head = torch.arange(kvh, device="cuda")[:, None, None]
    inside = torch.arange(bs, device="cuda")
    k = s["key_cache"][phys[..., None], inside, head].flatten(2, 3).float()   # (blocks, kvh, K * bs, hs)
    w = torch.einsum("nrkgd,nktd->nkrgt", q, k) / math.sqrt(hs)
    del k
    key = torch.where(some[..., None], best[..., None] * bs + inside, 1 << 30).flatten(2)
    seen = key[:, :, None, None] <= pos[:, None, :, None, None]
    w = w.masked_fill(~seen, -math.inf)
    most = w.amax(4, keepdim=True)
    w = torch.exp(w - torch.where(most == -math.inf, 0.0, most))
    total = w.sum(4, keepdim=True)
    v = s["value_cache"][phys[..., None], inside, head].flatten(2, 3).float()
    o = torch.einsum("nkrgt,nktd->nrkgd", w, v) / total.permute(0, 2, 1, 3, 4)
    lse = (most + torch.log(total))[..., 0].permute(0, 2, 1, 3).flatten(2)    # (blocks, R, nh)
    to = torch.where(there, rows, n).flatten()
    out = s["query"].new_empty(n + 1, nh * hs).index_copy(0, to, o.flatten(2).flatten(0, 1).to(s["query"].dtype))[:n]
    lse = lse.new_empty(n + 1, nh).index_copy(0, to, lse.flatten(0, 1))[:n]
    sel = torch.where(some, best, -1).int()
    sel = sel.new_empty(n + 1, kvh, K).index_copy(0, to, sel.repeat_interleave(R, 0))[:n]
    return [sel, out, lse]


# ---- what a pass cannot do without -----------------------------------------------------------


def work(case):
    if case["op"] == "rotate":
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["head_size"]
        return {"bytes": 4 * values + 4 * case["tokens"], "flops": 8 * values}
    past, q = _lengths(case, 0)
    bs, n = case["block_size"], len(q)
    rows = int(_cum(q)[-1])
    if case["op"] == "tables":
        rows = -(-rows // 64) * 64
        held = -(-past // bs)
        need = np.where(q > 0, -(-(past + np.maximum(q, 0)) // bs), 0)
        moved = int(np.maximum(need - held, 0).sum() + held[q < 0].sum())
        touched = int(np.where(q > 0, need - past // bs, 0).sum())
        return {"bytes": 4 * (5 * n + 2 * rows + 2 * moved + touched), "flops": 4 * n + 4 * rows}
    kvh, hs = case["kv_heads"], case["head_size"]
    if case["op"] == "bounds":
        touched = int((-(-(past + q) // bs) - past // bs).sum())
        values = rows * kvh * hs
        return {"bytes": 2 * values + touched * kvh * hs * 2 + 4 * (touched + 2 * n), "flops": 2 * values}
    nh, K, R = case["heads"], case["top_k"], case["query_block"]
    pages = -(-(past + q) // bs)
    blocks = -(-q // R)
    seen = np.minimum(pages, K)
    read = np.minimum(blocks * seen, pages)                 # pages of the cache read, each once
    data = read * bs * kvh * hs * 4 + pages * kvh * 2 * hs + 4 * pages + q * (2 * nh * hs * 2 + 4 * nh + 4 * kvh * K)
    ops = q * nh * seen * bs * hs * 4 + blocks * kvh * pages * hs * 4
    return {"bytes": int(data.sum()), "flops": int(ops.sum())}


# ---- the definitions in 64 bits --------------------------------------------------------------


def exact(case, seed):
    if case["op"] in ("tables", "bounds"):
        return None  # whole numbers only
    s = prepare(case, seed)
    return _exact_rotate(s) if case["op"] == "rotate" else _exact_sparse(s)


def _exact_rotate(s):
    c = s["case"]
    hs, d = c["head_size"], c["rotary"]
    half = d // 2
    freq = np.array([1e6 ** (-2.0 * u / d) for u in range(half)]).astype(np.float32) if d else np.zeros(0, np.float32)
    angle = torch.from_numpy((s["positions"].cpu().numpy().astype(np.float32)[:, None] * freq).astype(np.float64)).cuda()
    outs = []
    for x, heads, w in ((s["query"], c["heads"], s["q_weight"]), (s["key"], c["kv_heads"], s["k_weight"])):
        x = x.double().reshape(-1, heads, hs)
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / hs + 1e-6).sqrt() * w.double()
        if d:
            y = x.clone()
            for u in range(half):
                i, j = (2 * u, 2 * u + 1) if c["interleaved"] else (u, u + half)
                co, si = angle[:, None, u].cos(), angle[:, None, u].sin()
                y[..., i] = x[..., i] * co - x[..., j] * si
                y[..., j] = x[..., j] * co + x[..., i] * si
            x = y
        outs.append(x.reshape(len(x), -1))
    return outs


def _exact_sparse(s):
    """Request by request over its whole history, pages that are not selected masked out."""
    c = s["case"]
    nh, kvh, hs, bs, K, R = (c[k] for k in ("heads", "kv_heads", "head_size", "block_size", "top_k", "query_block"))
    G = nh // kvh
    cum, past = s["cum"].tolist(), s["past"].tolist()
    out = torch.empty(cum[-1], nh * hs, dtype=torch.float64, device="cuda")
    lse = torch.empty(cum[-1], nh, dtype=torch.float64, device="cuda")
    scale = s["scale"].cpu().numpy()
    for b in range(len(past)):
        q_len = cum[b + 1] - cum[b]
        if q_len == 0:
            continue
        total = past[b] + q_len
        n_pages = (total + bs - 1) // bs
        table = s["block_table"][b, :n_pages].long()
        bounds = s["bounds"][table].double()                                  # (pages, kvh, 2, hs)
        k_all, v_all = s["key_cache"][table].flatten(0, 1)[:total], s["value_cache"][table].flatten(0, 1)[:total]
        q_all = s["query"][cum[b]: cum[b + 1]].reshape(q_len, nh, hs)
        n_blocks = (q_len + R - 1) // R
        take = torch.zeros(n_blocks, kvh, n_pages, dtype=torch.bool, device="cuda")
        q_host = q_all.float().cpu().numpy()
        codes = np.zeros((2, n_blocks, kvh, hs), dtype=np.int64)
        for j in range(n_blocks):
            for g in range(kvh):
                x = q_host[j * R: (j + 1) * R, g * G: (g + 1) * G].reshape(-1, hs) * scale[g]
                top = np.float32(np.abs(x).max())
                if top > np.float32(1e-30):
                    t = np.rint(x * (np.float32(4095) / top)).astype(np.int64)
                    p, m = np.where(t > 0, t, 0).sum(0), np.where(t < 0, -t, 0).sum(0)
                    big = max(p.max(), m.max(), 1)
                    codes[0, j, g], codes[1, j, g] = (510 * p + big) // (2 * big), (510 * m + big) // (2 * big)
        codes = torch.from_numpy(codes).cuda().double()
        score = torch.einsum("jgd,pgd->jgp", codes[0], bounds[:, :, 1]) - torch.einsum("jgd,pgd->jgp", codes[1], bounds[:, :, 0])
        for j in range(n_blocks):
            last = (past[b] + min(q_len, (j + 1) * R) - 1) // bs
            own_page = (past[b] + j * R) // bs
            # a whole number per page that orders by score, then by index
            order = score[j, :, : last + 1].long() * (1 << 20) - torch.arange(last + 1, device="cuda")
            order[:, own_page:] = 1 << 60
            order[:, 0] = 1 << 60
            top = torch.topk(order, min(K, last + 1), dim=1).indices
            take[j].scatter_(1, top, True)
        of_row = torch.arange(q_len, device="cuda") // R
        step = max(1, min(q_len, (1 << 27) // (G * total)))
        for g in range(kvh):
            kg, vg = k_all[:, g].double(), v_all[:, g].double()
            for r0 in range(0, q_len, step):
                qg = q_all[r0: r0 + step, g * G: (g + 1) * G].double()
                ok = take[of_row[r0: r0 + step], g].repeat_interleave(bs, 1)[:, :total]
                ok = ok & (torch.arange(total, device="cuda") <= past[b] + r0 + torch.arange(len(qg), device="cuda")[:, None])
                w = (qg @ kg.T) / math.sqrt(hs)
                w.masked_fill_(~ok[:, None], -math.inf)
                z = torch.logsumexp(w, 2)
                o = torch.exp(w - z[..., None]) @ vg
                at = slice(cum[b] + r0, cum[b] + r0 + len(qg))
                out[at, g * G * hs: (g + 1) * G * hs] = o.flatten(1)
                lse[at, g * G: (g + 1) * G] = z
    return [None, out, lse]
