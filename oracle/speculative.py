"""Plain definitions of the speculative-decoding operators, element by element in numpy
(binary64 where values are computed), written from the formulas alone."""
from __future__ import annotations

import math

import numpy as np

NODES = 64


# --------------------------------------------------------------------------- numbers
def bf16(x):
    """Round float64 values to bfloat16 (nearest even), as float64; via f32, which holds a
    bf16 tie exactly, so only values that f32 itself rounds onto a tie could differ."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32) << 16
    return r.astype(np.uint32).view(np.float32).astype(np.float64)


def e4m3_value(code):
    """The value of e4m3 codes (uint8): sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    c = np.asarray(code, dtype=np.int64)
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(s == 1, -v, v)


_E4M3 = e4m3_value(np.arange(127))  # 0 .. 448, rising


def e4m3_code(x):
    """The nearest e4m3 code of finite x, |x| <= 464; ties to the even code."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.clip(np.searchsorted(_E4M3, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _E4M3[lo], _E4M3[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


# --------------------------------------------------------------------------- the cache
def offset(which, bytes_, H, D, block, page, head, token, d):
    """Element offset of (page, head, token of the page, d), from the layout's description."""
    base = ((page * H + head) * block + token // 16 * 16) * D
    t = token % 16
    if which == "k":
        e = 8 if bytes_ == 2 else 16
        p = [q for q in range(16) if (q & 3) | ((q >> 3) & 1) << 2 | ((q >> 2) & 1) << 3 == t][0]
        c, g, j = d // (4 * e), d % (4 * e) // e, d % e
        return base + ((c * 4 + g) * 16 + p) * e + j
    u = 1 if bytes_ == 2 else 2
    c, uu, m = d // (16 * u), d % (16 * u) // 16, d % 16
    return base + (((c * 2 + t // 8) * 16 + m) * u + uu) * 8 + t % 8


def offsets(which, bytes_, block, D):
    """offset() of every (token, d) of one head's page, as an array [block, D]."""
    return np.array([[offset(which, bytes_, 1, D, block, 0, 0, t, d) for d in range(D)] for t in range(block)])


def rows(cache, which, block, D, bytes_, table, n):
    """The first n tokens' raw rows [n, H, D] of a request with these pages, from a cache
    [pages, H, block, D] of raw elements; a page outside the cache gives zeros."""
    H = cache.shape[1]
    at = offsets(which, bytes_, block, D)
    out = np.zeros((n, H, D), dtype=cache.dtype)
    for pos in range(n):
        page = int(table[pos // block]) if pos // block < len(table) else -1
        if 0 <= page < cache.shape[0]:
            out[pos] = cache[page].reshape(H, block * D)[:, at[pos % block]]
    return out


def there(table, pages, block, n):
    """Which of the first n tokens lie in a page of the cache."""
    return np.array([pos // block < len(table) and 0 <= table[pos // block] < pages for pos in range(n)], dtype=bool)


# --------------------------------------------------------------------------- operators
def step_plan(ctx, new, owned, table, free, head, T, block, parents=None):
    R, width = table.shape
    table = table.copy()
    q_start, kv, slots = [0], [], np.full(T, -1, dtype=np.int64)
    pos_out, mask_out, owned_out = np.zeros(T, np.int64), np.zeros(T, np.uint64), owned.copy()
    at = max(head, 0)
    left = len(free) if head >= 0 else 0
    pages_asked = tokens_asked = 0
    for r in range(R):
        c, n, o = max(int(ctx[r]), 0), max(int(new[r]), 0), max(int(owned[r]), 0)
        owned_out[r] = o
        want = -(-(c + n) // block)
        need = max(0, want - o) if want <= width else 0
        tokens_asked += n
        room = tokens_asked <= T or (n == 0 and need == 0)
        served = want <= width and room and (need == 0 or (head >= 0 and head + pages_asked + need <= left))
        if served:
            for j in range(need):
                table[r, o + j] = free[head + pages_asked + j]
            owned_out[r] = o + need
            if need:
                at = head + pages_asked + need
        pages_asked += need
        first = q_start[-1]
        masks, depth = [], []
        for i in range(n):
            t = first + i
            if t >= T:
                break
            pos = c + i
            if served:
                slots[t] = int(table[r, pos // block]) * block + pos % block
            pos_out[t] = pos
            if parents is not None and n <= NODES:
                p = int(parents[t])
                if not 0 <= p < i:
                    p = -1
                masks.append((masks[p] if p >= 0 else 0) | (1 << i))
                depth.append(depth[p] + 1 if p >= 0 else 0)
                mask_out[t], pos_out[t] = masks[i], c + depth[i]
        kv.append(c + n if served else 0)
        q_start.append(min(first + n, T))
    return (np.array(q_start), np.array(kv), slots, pos_out, mask_out, owned_out, head if at < head or head < 0 else at,
            table)


def rotate(x, cos_sin, positions):
    """float64 rows [T, H, D], the first rot elements rotated in pairs (d, d + rot/2)."""
    x = np.array(x, dtype=np.float64)
    h = cos_sin.shape[1] // 2
    for t in range(x.shape[0]):
        row = cos_sin[min(max(int(positions[t]), 0), len(cos_sin) - 1)].astype(np.float64)
        a, b = x[t, :, :h].copy(), x[t, :, h:2 * h].copy()
        x[t, :, :h] = a * row[:h] - b * row[h:]
        x[t, :, h:2 * h] = b * row[:h] + a * row[h:]
    return x


def attention(q, k, v, ok, n, mask, scale):
    """One request and cache head: q [n, G, D] of its tokens, k, v [len, D], ok [len] (the key is
    there), mask: None (a chain) or the tokens' words.  Returns out [n, G, D], lse [n, G]."""
    length, G = len(k), q.shape[1]
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -math.inf)
    for i in range(n):
        sees = ok.copy()
        for pos in range(length):
            j = pos - (length - n)
            if j >= 0:
                sees[pos] &= bool(int(mask[i]) >> j & 1) if mask is not None and n <= NODES else j <= i
        if not sees.any():
            continue
        for g in range(G):
            s = scale * (k[sees] @ q[i, g])
            top = s.max()
            w = np.exp(s - top)
            lse[i, g] = top + math.log(w.sum())
            with np.errstate(invalid="ignore"):
                out[i, g] = (w / w.sum()) @ v[sees]
    return out, lse


def verify(logits, draft, parents, q_start, width=NODES):
    """logits float64 [T, V] -> accepted, path, next, target."""
    with np.errstate(invalid="ignore"):
        target = np.array([int(np.argmax(np.where(np.isnan(x), np.inf, x) if not np.isnan(x).any() else np.isnan(x)))
                           for x in logits], dtype=np.int64)
    R = len(q_start) - 1
    accepted, path, nxt = np.zeros(R, np.int64), np.full((R, width), -1, np.int64), np.full(R, -1, np.int64)
    for r in range(R):
        a, b = q_start[r], q_start[r + 1]
        n = b - a
        if n > NODES:
            accepted[r], nxt[r] = n, target[b - 1]
            continue
        cur, count = (0 if n else -1), 0
        while cur >= 0:
            if count < width:
                path[r, count] = cur
            count += 1
            want = target[a + cur]
            fits = [c for c in range(cur + 1, n) if parents[a + c] == cur and draft[a + c] == want]
            if not fits:
                nxt[r] = want
                break
            cur = fits[0]
        accepted[r] = count
    return accepted, path, nxt, target


def commit_moves(accepted, path, ctx, kv, table, pages, block):
    """[(request, from page, from token, to page, to token)], and the new context lengths."""
    moves, out = [], []
    for r in range(len(ctx)):
        c = max(int(ctx[r]), 0)
        n = max(int(kv[r]) - c, 0)
        count = min(max(int(accepted[r]), 0), n)
        if n <= NODES:
            count = min(count, path.shape[1])  # further nodes are not known
        out.append(c + count)
        if n > NODES:
            continue
        for i in range(count):
            p = int(path[r, i])
            if not i < p < n:
                continue
            a, b = c + p, c + i
            if max(a, b) // block >= table.shape[1]:
                continue
            pa, pb = int(table[r, a // block]), int(table[r, b // block])
            if 0 <= pa < pages and 0 <= pb < pages:
                moves.append((r, pa, a % block, pb, b % block))
    return moves, np.array(out)
