"""Plain numpy statements of the operators around the attention call, for their tests: whole
numbers as they are defined, the rest in 64 bits."""
from __future__ import annotations

import numpy as np


def block_tables(past, q, held, table, ring, state, bs, num_tokens):
    """What pa_build_block_tables writes, request by request."""
    past, q, held = (np.asarray(v, np.int64) for v in (past, q, held))
    table, ring, (head, count) = table.copy(), ring.copy(), (int(v) for v in state)
    B, cap, width = len(past), len(ring), table.shape[1]
    rows = np.maximum(q, 0)
    need = np.where(q > 0, -(-(past + rows) // bs), 0)
    grow = np.maximum(need - held, 0)
    back = np.where(q < 0, held, 0)
    error = 0
    if ((past < 0) | (q < -1) | (held < 0) | (held > width) | (need > width)).any() or rows.sum() > num_tokens or \
            not 0 <= head < cap or not 0 <= count <= cap or count + back.sum() > cap:
        error = 1
    elif grow.sum() > count:
        error = 16
    slots, positions = np.full(num_tokens, -1), np.full(num_tokens, -1)
    if error:
        return dict(cum=np.zeros(B + 1, int), slots=slots, positions=positions, held=held, state=[head, count],
                    error=error, table=table, ring=ring)
    new_held, at, tail = held.copy(), head, head + count
    cum = np.concatenate([[0], np.cumsum(rows)])
    for b in range(B):
        for col in range(held[b], held[b] + grow[b]):
            table[b, col] = ring[at % cap]
            at += 1
        new_held[b] = 0 if q[b] < 0 else held[b] + grow[b]
        p = past[b] + np.arange(rows[b])
        slots[cum[b]: cum[b + 1]] = table[b, p // bs].astype(np.int64) * bs + p % bs
        positions[cum[b]: cum[b + 1]] = p
    for b in range(B):
        for col in range(back[b]):
            ring[tail % cap] = table[b, col]
            tail += 1
    return dict(cum=cum, slots=slots, positions=positions, held=new_held,
                state=[at % cap, count - int(grow.sum()) + int(back.sum())], error=0, table=table, ring=ring)


def norm_rope(x, weight, eps, positions, rotary_dim, theta, interleaved):
    """(result, the magnitudes whose rounding errors it carries) of heads x (rows, heads, hs)."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    y, size = x.copy(), np.abs(x)
    d = rotary_dim
    if d:
        freq = np.array([float(theta) ** (-2.0 * u / d) for u in range(d // 2)]).astype(np.float32)
        angle = (positions.astype(np.float32)[:, None] * freq).astype(np.float64)[:, None]
        cos, sin = np.cos(angle), np.sin(angle)
        i, j = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
        y[..., i] = x[..., i] * cos - x[..., j] * sin
        y[..., j] = x[..., j] * cos + x[..., i] * sin
        size[..., i] = size[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return y, size


def key_codes(k, scale):
    """Codes of float32 keys (..., kvh, hs); NaN stays NaN."""
    with np.errstate(invalid="ignore", over="ignore"):
        return np.clip(np.rint(k.astype(np.float32) / scale), -127, 127)


def page_bounds(key_cache, bounds, scale, cum, past, table):
    """bounds (num_blocks, kvh, 2, hs) after a step whose rows are cum / past."""
    bounds = bounds.astype(np.int64).copy()
    bs = key_cache.shape[1]
    for b in range(len(past)):
        begin, end = int(past[b]), int(past[b]) + int(cum[b + 1] - cum[b])
        for page in range(begin // bs, -(-end // bs) if end > begin else 0):
            phys = table[b, page]
            k = key_codes(key_cache[phys, max(begin - page * bs, 0): min(end - page * bs, bs)], scale)
            lo = np.where(np.isnan(k), 127, k).min(0)
            hi = np.where(np.isnan(k), -127, k).max(0)
            if page * bs < begin:
                lo, hi = np.minimum(lo, bounds[phys, :, 0]), np.maximum(hi, bounds[phys, :, 1])
            bounds[phys, :, 0], bounds[phys, :, 1] = lo, hi
    return bounds


def query_codes(q, scale):
    """(positive, negative) 8-bit codes of the rows q (rows, hs) of one block and KV head."""
    with np.errstate(invalid="ignore", over="ignore"):
        x = q.astype(np.float32) * scale
    x = np.where(np.isfinite(x), x, np.float32(0))
    most = np.float32(np.abs(x).max()) if x.size else np.float32(0)
    if not most > np.float32(1e-30):
        return np.zeros(q.shape[1], int), np.zeros(q.shape[1], int)
    t = np.rint(x * (np.float32(4095) / most)).astype(np.int64)
    p, m = np.maximum(t, 0).sum(0), np.maximum(-t, 0).sum(0)
    big = max(p.max(), m.max())
    return (510 * p + big) // (2 * big), (510 * m + big) // (2 * big)


def select_pages(query, bounds, scale, cum, past, table, kvh, bs, top_k, R, sink, local, fill=-7):
    """selected (N, kvh, top_k); rows of no sequence hold `fill`. query (N, nh, hs) float32."""
    N, nh, hs = query.shape
    G = nh // kvh
    out = np.full((N, kvh, top_k), fill)
    for b in range(len(past)):
        q_len = int(cum[b + 1] - cum[b])
        for j0 in range(0, q_len, R):
            rows = slice(int(cum[b]) + j0, int(cum[b]) + min(j0 + R, q_len))
            own = (past[b] + j0) // bs
            n = (past[b] + min(j0 + R, q_len) - 1) // bs + 1
            for g in range(kvh):
                a, c = query_codes(query[rows, g * G: (g + 1) * G].reshape(-1, hs), scale[g])
                box = bounds[table[b, :n], g].astype(np.int64)
                score = box[:, 1] @ a - box[:, 0] @ c
                page = np.arange(n)
                always = (page < sink) | (page > own - local)
                order = np.lexsort((page, -score, ~always))
                take = np.sort(order[: top_k])
                out[rows, g] = np.concatenate([take, np.full(top_k - len(take), -1)])
    return out


def sparse_attention(query, key_cache, value_cache, cum, past, table, selected, scale, R):
    """(output (N, nh, hs), lse (N, nh), weighted |V| (N, nh, hs), the scores' rounding scale (N, nh)); rows of
    no sequence are NaN. float64 query (N, nh, hs) and caches."""
    N, nh, hs = query.shape
    bs, kvh = key_cache.shape[1:3]
    G = nh // kvh
    out, size = np.full((N, nh, hs), np.nan), np.full((N, nh, hs), np.nan)
    lse, mag = np.full((N, nh), np.nan), np.full((N, nh), np.nan)
    for b in range(len(past)):
        for j in range(int(cum[b + 1] - cum[b])):
            i, pos = int(cum[b]) + j, int(past[b]) + j
            first = int(cum[b]) + j // R * R
            for g in range(kvh):
                pages = [p for p in selected[first, g] if p >= 0]
                t = np.concatenate([[]] + [np.arange(p * bs, (p + 1) * bs) for p in pages]).astype(int)
                t = t[t <= pos]
                h = slice(g * G, (g + 1) * G)
                if len(t) == 0:
                    out[i, h], size[i, h], lse[i, h], mag[i, h] = 0, 0, -np.inf, 0
                    continue
                k, v = key_cache[table[b, t // bs], t % bs, g], value_cache[table[b, t // bs], t % bs, g]
                s = query[i, h] @ k.T * scale
                mag[i, h] = (np.abs(query[i, h]) @ np.abs(k.T)).max(1) * abs(scale)
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                total = p.sum(1, keepdims=True)
                out[i, h], size[i, h] = p @ v / total, p @ np.abs(v) / total
                lse[i, h] = (m + np.log(total))[:, 0]
    return out, lse, size, mag
