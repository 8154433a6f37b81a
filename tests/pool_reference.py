"""Plain numpy statements of the page operators and of the biased attention, for their tests: whole
numbers as they are defined, the rest in 64 bits."""
from __future__ import annotations

import numpy as np


def fork(parents, past, held, table, ring, state, bs, num_blocks, pinned=None):
    """What pa_fork_block_tables writes, row by row."""
    parents, past, held = (np.asarray(v, np.int64) for v in (parents, past, held))
    table, ring, (head, count) = np.asarray(table).copy(), np.asarray(ring).copy(), (int(v) for v in state)
    B, n, cap, width = len(past), len(parents), len(ring), table.shape[1]
    pinned = np.zeros(num_blocks, bool) if pinned is None else np.asarray(pinned) != 0
    need = -(-past // bs)
    error = 0
    if ((parents < -1) | (parents >= B)).any() or (past < 0).any() or ((held < 0) | (held > width)).any() or \
            not 0 <= head < cap or not 0 <= count <= cap:
        error = 1
    elif any(need[p] > held[p] for p in parents if p >= 0):
        error = 1
    pages = [[int(x) for x in table[b, : held[b] if 0 <= held[b] <= width else 0]] for b in range(B)]
    if any(not 0 <= x < num_blocks for row in pages for x in row):
        error |= 2
    refused = dict(past=np.zeros(n, int), held=np.zeros(n, int), table=np.full((n, width), -1), copies=np.full((n, 2), -1),
                   state=[head, count], ring=ring.copy())
    if error:
        return refused | dict(error=error)
    out = dict(past=np.array([past[p] if p >= 0 else 0 for p in parents], int), copies=np.full((n, 2), -1),
               table=np.full((n, width), -1))
    out["held"] = -(-out["past"] // bs)
    whole, last = set(), {}
    for b, p in enumerate(parents):
        if p < 0:
            continue
        full = int(past[p]) // bs
        whole.update(pages[p][:full])
        if past[p] % bs:
            last.setdefault(pages[p][full], []).append(b)
        out["table"][b, : need[p]] = pages[p][: need[p]]
    takers = sorted(b for x, rows in last.items() for b in rows if x in whole or pinned[x] or b != rows[0])
    gone = sorted({x for row in pages for x in row} - whole - set(last) - set(np.flatnonzero(pinned).tolist()))
    if count + len(gone) > cap:
        return refused | dict(error=1)
    if len(takers) > count:
        return refused | dict(error=16)
    for i, b in enumerate(takers):
        col, new = out["past"][b] // bs, ring[(head + i) % cap]
        out["copies"][i] = out["table"][b, col], new
        out["table"][b, col] = new
    for i, x in enumerate(gone):
        ring[(head + count + i) % cap] = x
    return out | dict(ring=ring, state=[(head + len(takers)) % cap, count - len(takers) + len(gone)], error=0)


def compact(held, table, ring, num_blocks, max_moves, pinned=None):
    """What pa_compact_block_tables writes."""
    held, table, ring = np.asarray(held, np.int64), np.asarray(table).copy(), np.asarray(ring).copy()
    pinned = np.zeros(num_blocks, bool) if pinned is None else np.asarray(pinned) != 0
    refused = dict(table=table.copy(), copies=np.full((max_moves, 2), -1), state=[0, 0], end=0, ring=ring.copy())
    if ((held < 0) | (held > table.shape[1])).any():
        good = (held >= 0) & (held <= table.shape[1])
        x = [v for b in np.flatnonzero(good) for v in table[b, : held[b]]]
        return refused | dict(error=1 | (2 if any(not 0 <= v < num_blocks for v in x) else 0))
    used = pinned.copy()
    for b in range(len(held)):
        for x in table[b, : held[b]]:
            if not 0 <= x < num_blocks:
                return refused | dict(error=2)
            used[x] = True
    holes = np.flatnonzero(~used)
    if len(holes) > len(ring):
        return refused | dict(error=1)
    movers = np.flatnonzero(used & ~pinned)[::-1]
    to, copies = np.arange(num_blocks), np.full((max_moves, 2), -1)
    for r in range(min(max_moves, len(movers), len(holes))):
        if holes[r] > movers[r]:
            break
        to[movers[r]] = holes[r]
        copies[r] = movers[r], holes[r]
        used[movers[r]], used[holes[r]] = False, True
    for b in range(len(held)):
        table[b, : held[b]] = to[table[b, : held[b]]]
    free = np.flatnonzero(~used)
    ring[: len(free)] = free
    return dict(table=table, copies=copies, state=[0, len(free)], end=int(np.flatnonzero(used).max(initial=-1)) + 1,
                ring=ring, error=0)


def key_range(past, q, j, window, first, prefix):
    """The keys [lo, hi) that row j of a sequence sees."""
    p = past + j
    lo = max(0, first if first is not None else 0, p - window + 1 if window else 0)
    hi = min(past + q, max(p + 1, prefix if prefix is not None else 0))
    return lo, max(lo, hi)


def biased_attention(query, key_cache, value_cache, cum, past, table, scale, softcap=0.0, slopes=None, window=0,
                     first_keys=None, prefix_lens=None):
    """(output (N, nh, hs), lse (N, nh), weighted |V| (N, nh, hs), the scores' rounding scale before the cap and the
    largest bias of a row (N, nh)); rows of no sequence are NaN. float64 query (N, nh, hs) and caches."""
    N, nh, hs = query.shape
    bs, kvh = key_cache.shape[1:3]
    G = nh // kvh
    out, size = np.full((N, nh, hs), np.nan), np.full((N, nh, hs), np.nan)
    lse, mag, far = np.full((N, nh), np.nan), np.full((N, nh), np.nan), np.zeros((N, nh))
    for b in range(len(past)):
        q_len = int(cum[b + 1] - cum[b])
        for j in range(q_len):
            i, pos = int(cum[b]) + j, int(past[b]) + j
            lo, hi = key_range(int(past[b]), q_len, j, window, None if first_keys is None else int(first_keys[i]),
                               None if prefix_lens is None else int(prefix_lens[b]))
            t = np.arange(lo, hi)
            for g in range(kvh):
                h = slice(g * G, (g + 1) * G)
                if len(t) == 0:
                    out[i, h], size[i, h], lse[i, h], mag[i, h] = 0, 0, -np.inf, 0
                    continue
                k, v = key_cache[table[b, t // bs], t % bs, g], value_cache[table[b, t // bs], t % bs, g]
                s = query[i, h] @ k.T * scale
                mag[i, h] = (np.abs(query[i, h]) @ np.abs(k.T)).max(1) * abs(scale)
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    bias = np.abs(pos - t) * np.asarray(slopes, np.float64)[h, None]
                    s, far[i, h] = s - bias, np.abs(bias).max(1)
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                total = p.sum(1, keepdims=True)
                out[i, h], size[i, h] = p @ v / total, p @ np.abs(v) / total
                lse[i, h] = (m + np.log(total))[:, 0]
    return out, lse, size, mag, far
