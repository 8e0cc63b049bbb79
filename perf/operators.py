"""Cases of the speculative-decoding operators: what is measured, in plain torch and through the package.

One decoding step over a paged K/V cache is five operators: step_plan (block tables, slot map,
positions and tree masks from the request lengths), kv_write (rotary embedding, K/V rows into the
cache), tree_attention (the step's tokens against cache and tree), tree_verify (greedy check of the
drafted tree against the logits) and kv_commit (accepted rows moved together).

The cache holds 16-token tiles in matrix-operand order.  A page of one head is block/16 tiles; for
2-byte elements a K tile is [D/32][4 g][16 p][8 e] with d = 32 c + 8 g + e and a V tile is
[D/16][2 o][16 m][8 i] with token 8 o + i, d = 16 c + m; for e4m3 a K tile is [D/64][4 g][16 p][16 e]
with d = 64 c + 16 g + e and a V tile [D/32][2 o][16 m][2 u][8 i] with d = 32 c + 16 u + m.  Place p of
a K tile holds the token with bits (p2, p3, p1, p0).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
MAX_NODES = 64
E4M3_MAX = 448.0


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one user, a small drafted tree: the call's latency
        dict(name="plan one tree", op="plan", requests=1, new=33, context=700, block=16, tree=True),
        # a full server: prompts' chunks of very different lengths, tens of thousands of tokens
        dict(name="plan prompt batch", op="plan", requests=512, new=256, context=30000, block=32, tree=False),
        # eight users' trees through one layer with wide heads and a partial rotary embedding
        dict(name="write trees bf16", op="write", tokens=128, kv_heads=4, group=6, head_dim=256, rot=64,
             cache="bf16", block=16),
        # an odd prompt chunk into an 8-bit cache
        dict(name="write prompt e4m3", op="write", tokens=8191, kv_heads=8, group=4, head_dim=128, rot=128,
             cache="e4m3", block=64),
        # one user, one token, short cache: latency
        dict(name="attend one token", op="attend", requests=1, nodes=1, context=1000, ragged=False, tree=True,
             kv_heads=4, group=6, head_dim=256, cache="bf16", block=16),
        # a batch of full trees over caches of all lengths
        dict(name="attend tree batch", op="attend", requests=16, nodes=64, context=8192, ragged=True, tree=True,
             kv_heads=8, group=4, head_dim=128, cache="bf16", block=32),
        # a few small trees over long 8-bit caches: the cache's bytes
        dict(name="attend long e4m3", op="attend", requests=4, nodes=8, context=131071, ragged=False, tree=True,
             kv_heads=8, group=4, head_dim=128, cache="e4m3", block=64),
        # prompt chunks on top of what the cache holds: the matrix cores
        dict(name="attend prompt chunk", op="attend", requests=2, nodes=2048, context=2048, ragged=False, tree=False,
             kv_heads=4, group=6, head_dim=256, cache="bf16", block=64),
        # one user's tree against the whole vocabulary
        dict(name="verify one tree", op="verify", requests=1, nodes=17, vocab=248320, logits="f32"),
        # a batch of trees
        dict(name="verify batch", op="verify", requests=32, nodes=16, vocab=248320, logits="bf16"),
        # one user, one layer's cache
        dict(name="commit one layer", op="commit", requests=1, nodes=17, context=1500, layers=1, kv_heads=8,
             head_dim=128, cache="bf16", block=16),
        # all sixteen attention layers of a batch in one call
        dict(name="commit all layers", op="commit", requests=64, nodes=64, context=900, layers=16, kv_heads=4,
             head_dim=256, cache="e4m3", block=32),
    ]


def _log(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "write", "attend", "attend", "verify", "commit"])
    block = rng.choice([16, 32, 64, 128])
    if op == "plan":
        tree = rng.random() < 0.5
        return dict(op=op, requests=_log(rng, 1, 512), new=_log(rng, 1, 64 if tree else 256),
                    context=_log(rng, 1, 30000), block=block, tree=tree)
    dim = rng.choice([64, 128, 256])
    heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 8])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 8191 * 8 * 128 * 3 // (heads * (group + 2) * dim)), kv_heads=heads,
                    group=group, head_dim=dim, rot=rng.choice([0, dim // 4, dim // 2, dim]), cache=cache, block=block)
    if op == "attend":
        tree = rng.random() < 0.75
        nodes = _log(rng, 1, 64 if tree else 2048)
        # tokens of cache over all requests: within the long listed case's bytes and the chunk's products
        most = min(4 * 131071 * 8 * 128 // (heads * dim), 144 * 2048 * 1024 * 256 // (heads * group * nodes * dim))
        requests = _log(rng, 1, max(1, min(64, most // 64)))
        return dict(op=op, requests=requests, nodes=nodes, context=_log(rng, 1, max(1, min(131071, most // requests))),
                    ragged=rng.random() < 0.6, tree=tree, kv_heads=heads, group=group, head_dim=dim, cache=cache,
                    block=block)
    if op == "verify":
        nodes = _log(rng, 1, 64)
        return dict(op=op, requests=_log(rng, 1, max(1, 512 // nodes)), nodes=nodes, vocab=_log(rng, 1000, 248320),
                    logits=rng.choice(["f32", "bf16"]) if nodes < 32 else "bf16")
    return dict(op=op, requests=_log(rng, 1, 64), nodes=_log(rng, 1, 64), context=_log(rng, 1, 900),
                layers=rng.choice([1, 4, 16]), kv_heads=min(heads, 4), head_dim=dim, cache=cache, block=block)


def _spread(count, most, least, power):
    """count lengths in [least, most], unevenly spread in a fixed order; the first is the longest."""
    return [int(least + (most - least) * (1.0 - (r * 0.6180339887498949) % 1.0) ** power) for r in range(count)]


def _lengths(case):
    """(context lengths, new lengths) of the requests, from the case alone."""
    R = case["requests"]
    if case["op"] == "plan":
        new = _spread(R, case["new"], 1, 1)
        return _spread(R, case["context"], 0, 2), new
    if case["op"] == "attend" and case["ragged"]:
        return _spread(R, case["context"], 0, 1), _spread(R, case["nodes"], 1, 1)
    return [case["context"]] * R, [case["nodes"]] * R


def _sum(v):
    return int(sum(v))


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _trees(rng, sizes, chain=0.5):
    """Parents of drafted trees: node 0 is the root, every other node's parent is an earlier node."""
    parents = []
    for n in sizes:
        i = np.arange(n)
        p = np.where(rng.random(n) < chain, i - 1, (rng.random(n) * np.maximum(i, 1)).astype(np.int64))
        parents.append(np.where(i == 0, -1, np.minimum(p, i - 1)))
    return np.concatenate(parents).astype(np.int32)


def _masks(parents, sizes):
    """Ancestor bits (the node's own among them) of every node, as int64."""
    out, at = [], 0
    for n in sizes:
        m = [0] * n
        for i in range(n):
            p = int(parents[at + i])
            m[i] = (m[p] if p >= 0 else 0) | (1 << i)
        out += m
        at += n
    return np.array(out, dtype=np.uint64).view(np.int64)


def _pool(g, lens, block, spare):
    """Block tables over a shuffled pool: int32 [R, widest], and the pool's size."""
    pages = [-(-n // block) for n in lens]
    total, wide = sum(pages) + spare, max(max(pages), 1)
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((len(lens), wide), dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = order[at:at + n]
        at += n
    return table, total


def _cache(g, shape, cache):
    """A filled cache of `shape` [..., pages, heads, block, D]: (codes, scales or None)."""
    x = _randn(g, shape, torch.bfloat16)
    if cache == "bf16":
        return x, None
    scale = torch.exp(0.25 * _randn(g, shape[:-1])) * (3.5 / E4M3_MAX)
    return (x * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g, rng, op = _gen(seed), np.random.default_rng(seed), case["op"]
    s = {"op": op, "block": case.get("block")}
    if op == "plan":
        ctx, new = _lengths(case)
        R, bs = len(ctx), case["block"]
        ctx = [max(0, c - int(rng.integers(0, 9))) for c in ctx]
        owned = [-(-c // bs) for c in ctx]
        s["table"], total = _pool(g, ctx, bs, 0)
        wide = max(-(-(c + n) // bs) for c, n in zip(ctx, new))
        table = torch.zeros((R, wide), dtype=torch.int32, device=DEV)
        table[:, :min(wide, s["table"].shape[1])] = s["table"][:, :wide]
        spare = sum(-(-(c + n) // bs) - o for c, n, o in zip(ctx, new, owned)) + 7
        s["table"] = table
        s["free"] = (torch.randperm(spare, generator=g, device=DEV) + total).to(torch.int32)
        s["head"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["ctx"], s["new"], s["owned"], s["tokens"] = _ints(ctx), _ints(new), _ints(owned), _sum(new)
        s["parents"] = torch.from_numpy(_trees(rng, new)).to(DEV) if case["tree"] else None
        return s
    if op == "write":
        T, H, G, D, bs = (case[k] for k in ("tokens", "kv_heads", "group", "head_dim", "block"))
        # the qkv layer's output: q, k and v are column ranges of its rows
        qkv = _randn(g, (T, (G + 2) * H * D), torch.bfloat16)
        s["q"] = qkv[:, :G * H * D].unflatten(1, (G * H, D))
        s["k"] = qkv[:, G * H * D:(G + 1) * H * D].unflatten(1, (H, D))
        s["v"] = qkv[:, (G + 1) * H * D:].unflatten(1, (H, D))
        pages = -(-T // bs) + 3
        first = int(rng.integers(0, bs))  # the chunk starts inside a page
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(T, device=DEV) + first
        s["slots"] = order[at // bs] * bs + at % bs
        s["positions"] = (at + int(rng.integers(0, 30000))).to(torch.int32)
        s["cos_sin"] = None
        if case["rot"]:
            h = case["rot"] // 2
            f = 1e6 ** (-torch.arange(h, dtype=torch.float64, device=DEV) / h)
            a = torch.arange(131072 // 2, dtype=torch.float64, device=DEV)[:, None] * f
            s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        s["q_out"] = torch.empty((T, G * H, D), dtype=torch.bfloat16, device=DEV)
        kind = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
        for n in "kv":
            s[n + "_cache"] = torch.zeros((pages, H, bs, D), dtype=torch.uint8, device=DEV).to(kind)
            s[n + "_scale"] = None if case["cache"] == "bf16" else torch.zeros((pages, H, bs), device=DEV)
        return s
    if op == "verify":
        R, n, V = case["requests"], case["nodes"], case["vocab"]
        sizes = [n] * R
        kind = torch.float32 if case["logits"] == "f32" else torch.bfloat16
        s["logits"] = _randn(g, (R * n, V), kind)
        parents = _trees(rng, sizes)
        tokens = rng.integers(0, V, R * n).astype(np.int32)
        # a good draft: two nodes in three carry what the model answers at their parent
        want = rng.integers(0, V, R * n).astype(np.int32)
        base = (np.arange(R * n) // n) * n
        tokens = np.where((rng.random(R * n) < 0.67) & (parents >= 0), want[base + np.maximum(parents, 0)], tokens)
        s["logits"][torch.arange(R * n, device=DEV), torch.from_numpy(want.astype(np.int64)).to(DEV)] = 9.0
        s["draft"], s["parents"] = torch.from_numpy(tokens.astype(np.int32)).to(DEV), torch.from_numpy(parents).to(DEV)
        s["q_start"] = _ints([n * r for r in range(R + 1)])
        return s
    ctx, new = _lengths(case)
    R, H, D, bs = len(ctx), case["kv_heads"], case["head_dim"], case["block"]
    lens = [c + n for c, n in zip(ctx, new)]
    s["table"], pages = _pool(g, lens, bs, 2)
    s["ctx"], s["kv_lens"], s["q_start"] = _ints(ctx), _ints(lens), _ints([0] + np.cumsum(new).tolist())
    s["widest"], s["longest"] = max(new), max(lens)
    lead = (case["layers"],) if op == "commit" else ()
    for n in "kv":
        s[n + "_cache"], s[n + "_scale"] = _cache(g, lead + (pages, H, bs, D), case["cache"])
    if op == "attend":
        G, T = case["group"], sum(new)
        s["q"] = (2.0 * _randn(g, (T, G * H, D))).to(torch.bfloat16)
        s["mask"] = torch.from_numpy(_masks(_trees(rng, new), new)).to(DEV) if case["tree"] else None
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((T, G * H), device=DEV)
        return s
    path = np.full((R, MAX_NODES), -1, dtype=np.int32)  # accepted paths: increasing nodes from the root
    count = np.zeros(R, dtype=np.int32)
    for r, n in enumerate(new):
        k = 1 + int(rng.integers(0, min(n, 12)))
        path[r, :k] = np.concatenate([[0], 1 + np.sort(rng.permutation(n - 1)[:k - 1])]) if n > 1 else 0
        count[r] = k
    s["path"], s["accepted"] = torch.from_numpy(path).to(DEV), torch.from_numpy(count).to(DEV)
    s["ctx_out"] = torch.empty(R, dtype=torch.int32, device=DEV)
    return s


# --------------------------------------------------------------------------- plain forms
def _k_tiles(cache):
    """The K cache [..., heads, block, D] as [..., heads, block/16, D/w, 4, 16, e]: place at dim -2."""
    e = 8 if cache.dtype == torch.bfloat16 else 16
    return _bits(cache).unflatten(-2, (-1, 16)).flatten(-2).unflatten(-1, (cache.shape[-1] // (4 * e), 4, 16, e))


def _v_tiles(cache):
    """The V cache as [..., heads, block/16, D/w, 2, 16, u, 8]: token 8 o + i at dims -4 and -1."""
    u = 1 if cache.dtype == torch.bfloat16 else 2
    return _bits(cache).unflatten(-2, (-1, 16)).flatten(-2).unflatten(-1, (cache.shape[-1] // (16 * u), 2, 16, u, 8))


def _place(token):
    return token % 4 + token // 8 % 2 * 4 + token // 4 % 2 * 8


def _bits(cache):
    return cache.view(torch.int16 if cache.dtype == torch.bfloat16 else torch.uint8)


def _values(bits):
    return bits.view(torch.bfloat16 if bits.dtype == torch.int16 else torch.float8_e4m3fn).float()


def _k_rows(cache, slots, block, rows=None):
    """Raw rows [n, ..., heads, D] of the K cache at `slots` [n], or with `rows` writes them."""
    t, b, i = _k_tiles(cache), slots // block, slots % block
    at = (b, slice(None), i // 16, slice(None), slice(None), _place(i % 16))
    at = at if t.dim() == 7 else (slice(None),) + at
    if rows is None:
        return t[at].flatten(-3)
    t[at] = rows.unflatten(-1, t.shape[-4:-2] + t.shape[-1:])


def _v_rows(cache, slots, block, rows=None):
    t, b, i = _v_tiles(cache), slots // block, slots % block
    at = (b, slice(None), i // 16, slice(None), i % 16 // 8, slice(None), slice(None), i % 8)
    at = at if t.dim() == 8 else (slice(None),) + at
    if rows is None:
        return t[at].transpose(-1, -2).flatten(-3)
    t[at] = rows.unflatten(-1, (t.shape[-5], t.shape[-2], 16)).transpose(-1, -2)


def _ancestors(parents, first, i):
    """Bits of each node's ancestors and its own, by doubling the reach; invalid parents are roots."""
    up = torch.where((parents >= 0) & (parents < i), parents, -1)
    bits = torch.ones_like(i) << (i & 63)
    for _ in range(6):
        to = first + up.clamp_min(0)
        bits = torch.where(up >= 0, bits | bits[to], bits)
        up = torch.where(up >= 0, up[to], up)
    return bits


def _plan_plain(s):
    ctx, new, owned, bs, T = s["ctx"].long(), s["new"].long(), s["owned"].long(), s["block"], s["tokens"]
    table, free, head = s["table"], s["free"].long(), s["head"].long()
    want = (ctx + new + bs - 1) // bs
    fits = want <= table.shape[1]
    need = torch.where(fits, (want - owned).clamp_min(0), 0)
    off = need.cumsum(0) - need
    served = fits & ((need == 0) | (head + off + need <= free.numel()))
    taken = torch.where(served, need, 0)
    q_start = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)]).clamp_max(T)
    col = torch.arange(table.shape[1], device=table.device)
    j = col - owned[:, None]
    fresh = free[(head + off[:, None] + j).clamp(0, free.numel() - 1)]
    table.copy_(torch.where((j >= 0) & (j < taken[:, None]), fresh, table.long()))
    t = torch.arange(T, device=table.device)
    r = torch.searchsorted(q_start[1:], t, right=True)
    there = r < new.numel()
    r = r.clamp_max(new.numel() - 1)
    i = t - q_start[r]
    pos = ctx[r] + i
    ok = there & served[r]
    slots = torch.where(ok, table[r, torch.where(ok, pos // bs, 0)].long() * bs + pos % bs, -1)
    mask = None
    if s["parents"] is not None:
        mask = _ancestors(s["parents"].long(), q_start[r], i)
        depth = ((mask[:, None] >> torch.arange(64, device=t.device)) & 1).sum(1) - 1
        tree = new[r] <= MAX_NODES
        pos = torch.where(tree, ctx[r] + depth, pos)
        mask = torch.where(there & tree, mask, 0)
    pos = torch.where(there, pos, 0)
    return (q_start.int(), torch.where(served, ctx + new, 0).int(), slots, pos.int(), mask,
            (owned + taken).int(), (head + taken.sum()).int(), table)


def _rotated(x, cos_sin, positions):
    if cos_sin is None:
        return x
    h = cos_sin.shape[1] // 2
    c, n = cos_sin[positions.long()][:, None, :].split(h, -1)
    f = x.float()
    a, b = f[..., :h], f[..., h:2 * h]
    return torch.cat([a * c - b * n, b * c + a * n, f[..., 2 * h:]], -1).to(torch.bfloat16)


def _e4m3(x):
    top = x.float().abs().amax(-1)
    scale = top / torch.full_like(top, E4M3_MAX)  # a tensor: torch multiplies by a number's reciprocal instead
    code = torch.where(scale[..., None] > 0, x.float() / scale[..., None], 0.0)
    return code.to(torch.float8_e4m3fn), scale


def _write_plain(s):
    bs, slots = s["block"], s["slots"]
    s["q_out"].copy_(_rotated(s["q"], s["cos_sin"], s["positions"]))
    k, v = _rotated(s["k"], s["cos_sin"], s["positions"]), s["v"]
    if s["k_scale"] is not None:
        k, ks = _e4m3(k)
        v, vs = _e4m3(v)
        s["k_scale"][slots // bs, :, slots % bs] = ks
        s["v_scale"][slots // bs, :, slots % bs] = vs
    _k_rows(s["k_cache"], slots, bs, _bits(k.contiguous()))
    _v_rows(s["v_cache"], slots, bs, _bits(v.contiguous()))
    return s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _attend_plain(s):
    bs, q, table, L, n = s["block"], s["q"], s["table"].long(), s["longest"], s["widest"]
    H, D = s["k_cache"].shape[1], s["k_cache"].shape[3]
    R, T, G = table.shape[0], q.shape[0], q.shape[1] // H
    # pages [R, pages, heads, tiles, ...] laid out as rows [R, heads, tokens, D]
    place = _place(torch.arange(16, device=q.device))
    k = _k_tiles(s["k_cache"])[table].index_select(6, place).permute(0, 2, 1, 3, 6, 4, 5, 7)
    v = _v_tiles(s["v_cache"])[table].permute(0, 2, 1, 3, 5, 8, 4, 7, 6)
    k = _values(k.contiguous()).reshape(R, H, -1, D)
    v = _values(v.contiguous()).reshape(R, H, -1, D)
    if s["k_scale"] is not None:
        k = k * s["k_scale"][table].transpose(1, 2).reshape(R, H, -1, 1)
        v = v * s["v_scale"][table].transpose(1, 2).reshape(R, H, -1, 1)
    k, v = k[:, :, :L], v[:, :, :L].contiguous()
    first, kv = s["q_start"][:-1].long(), s["kv_lens"].long()
    count = s["q_start"][1:].long() - first
    node = torch.arange(n, device=q.device)
    row = (first[:, None] + node).clamp_max(T - 1)                      # [R, n]
    qp = q[row].float().reshape(R, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, n * G, D)
    score = torch.matmul(qp * D ** -0.5, k.transpose(2, 3).contiguous())
    key = torch.arange(k.shape[2], device=q.device)
    j = key - (kv - count)[:, None]                                     # [R, L]: the node a key is, < 0: context
    if s["mask"] is not None:
        seen = ((s["mask"][row][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1).bool()
    else:
        seen = j[:, None, :] <= node[:, None]
    seen = ((j < 0)[:, None, :] | seen) & (key < kv[:, None])[:, None, :]  # [R, n, L]
    score = torch.where(seen[:, None, :, None, :], score.unflatten(2, (n, G)), -math.inf).flatten(2, 3)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    t = torch.arange(T, device=q.device)
    r = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    i = t - first[r]
    o = o.reshape(R, H, n, G, D)[r, :, i].reshape(T, H * G, D).to(torch.bfloat16)
    return o, lse.reshape(R, H, n, G)[r, :, i].reshape(T, H * G)


def _verify_plain(s):
    x = s["logits"].float()
    V, R = x.shape[1], s["q_start"].numel() - 1
    at = torch.arange(V, device=x.device)
    target = torch.where(x == x.amax(1, keepdim=True), at, V).amin(1)
    first = s["q_start"][:-1].long()
    count = s["q_start"][1:].long() - first
    i = torch.arange(MAX_NODES, device=x.device)
    there = i < count[:, None]
    t = (first[:, None] + i).clamp_max(x.shape[0] - 1)                  # [R, 64]
    up, draft = s["parents"].long()[t], s["draft"].long()[t]
    up = torch.where((up >= 0) & (up < i) & there, up, -1)
    fits = (up >= 0) & (draft == torch.gather(target[t], 1, up.clamp_min(0)))
    twin = fits[:, None, :] & (up[:, None, :] == up[:, :, None]) & (i[None, None, :] < i[None, :, None])
    good = (fits & ~twin.any(2)) | ((i == 0) & there)                   # as its parent's choice; node 0 is given
    to = torch.where(i == 0, 0, up)
    for _ in range(6):
        good = good & torch.where(to >= 0, torch.gather(good, 1, to.clamp_min(0)), False)
        to = torch.where(to >= 0, torch.gather(to, 1, to.clamp_min(0)), -1)
    accepted = good.sum(1)
    path = torch.where(good, i, MAX_NODES).sort(1).values
    last = torch.where(good, i, 0).amax(1)
    nxt = torch.gather(target[t], 1, last[:, None]).squeeze(1)
    return (accepted.int(), torch.where(path < MAX_NODES, path, -1).int(), nxt.int(), target.int())


def _commit_plain(s):
    bs, table, path = s["block"], s["table"].long(), s["path"].long()
    ctx = s["ctx"].long()
    i = torch.arange(MAX_NODES, device=path.device)
    go = i < s["accepted"][:, None]
    src = (ctx[:, None] + torch.where(go, path, 0))                     # the others rewrite the root's row onto itself
    dst = (ctx[:, None] + torch.where(go, i, 0))
    src, dst = (torch.gather(table, 1, p // bs) * bs + p % bs for p in (src, dst))
    src, dst = src.reshape(-1), dst.reshape(-1)
    _k_rows(s["k_cache"], dst, bs, _k_rows(s["k_cache"], src, bs))
    _v_rows(s["v_cache"], dst, bs, _v_rows(s["v_cache"], src, bs))
    if s["k_scale"] is not None:
        for c in (s["k_scale"], s["v_scale"]):
            c[:, dst // bs, :, dst % bs] = c[:, src // bs, :, src % bs]
    s["ctx_out"].copy_(ctx + s["accepted"])
    return s["ctx_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def run(s):
    op = s["op"]
    if not own:
        return {"plan": _plan_plain, "write": _write_plain, "attend": _attend_plain, "verify": _verify_plain,
                "commit": _commit_plain}[op](s)
    import quantized_gemv_gemm_amd as tl
    if op == "plan":
        got = tl.step_plan(s["ctx"], s["new"], s["owned"], s["table"], s["free"], s["head"], s["tokens"], s["block"],
                           parents=s["parents"])
        return (*got, s["table"])
    if op == "write":
        tl.kv_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"],
                    v_scale=s["v_scale"], q=s["q"], positions=s["positions"], cos_sin=s["cos_sin"], q_out=s["q_out"])
        return s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if op == "attend":
        return tl.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_lens"],
                                 tree_mask=s["mask"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                 max_nodes=s["widest"], out=s["out"], lse=s["lse"])
    if op == "verify":
        return tl.tree_verify(s["logits"], s["draft"], s["parents"], s["q_start"])
    tl.kv_commit(s["accepted"], s["path"], s["ctx"], s["kv_lens"], s["table"], s["k_cache"], s["v_cache"],
                 k_scale=s["k_scale"], v_scale=s["v_scale"], ctx_out=s["ctx_out"])
    return s["ctx_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


# --------------------------------------------------------------------------- work and the exact values
def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _lengths(case)
        T, bs = _sum(new), case["block"]
        pages = sum(-(-(c + n) // bs) - c // bs for c, n in zip(ctx, new))  # pages the tokens touch
        return {"bytes": 12 * len(ctx) + 12 * len(ctx) + 8 * pages + T * (24 if case["tree"] else 12), "flops": T}
    if op == "verify":
        size = 4 if case["logits"] == "f32" else 2
        T = case["requests"] * case["nodes"]
        return {"bytes": T * (case["vocab"] * size + 12) + case["requests"] * 268, "flops": T * case["vocab"]}
    H, D = case["kv_heads"], case["head_dim"]
    row = H * (D * 2 if case["cache"] == "bf16" else D + 4)                 # one token of K or of V
    if op == "write":
        T, G = case["tokens"], case["group"]
        return {"bytes": T * (2 * D * H * (G + 2) + 2 * D * H * G + 2 * row + 12 + 4 * case["rot"]),
                "flops": 3 * T * H * ((G + 1) * case["rot"] + (0 if case["cache"] == "bf16" else 2 * D))}
    ctx, new = _lengths(case)
    if op == "attend":
        G, T = case["group"], _sum(new)
        pairs = sum(n * c + (n * (n + 1) // 2 if not case["tree"] else n * n) for c, n in zip(ctx, new))
        return {"bytes": 2 * row * (_sum(ctx) + T) + 4 * T * G * H * D + 4 * T * G * H + 8 * T * case["tree"],
                "flops": 4 * pairs * H * G * D}
    moved = min(case["nodes"], 12) / 2 * case["requests"]                   # the mean accepted length, less the root
    return {"bytes": case["layers"] * 4 * row * max(moved, 1) + case["requests"] * 280, "flops": 0}


def _untile(cache, scale, pages):
    """(a page list's) tokens [len(pages) * block, heads, D] in 64 bits, element by element from the layout."""
    H, bs, D = cache.shape[-3:]
    e, u = (8, 1) if cache.dtype == torch.bfloat16 else (16, 2)
    flat = cache.reshape(-1, H, bs * D)[pages]
    tok, d = torch.meshgrid(torch.arange(bs, device=DEV), torch.arange(D, device=DEV), indexing="ij")
    tile, t = tok // 16 * (16 * D), tok % 16
    p = (t & 3) | (t & 8) >> 1 | (t & 4) << 1
    k_at = tile + d // (4 * e) * (64 * e) + d % (4 * e) // e * (16 * e) + p * e + d % e
    v_at = tile + d // (16 * u) * (256 * u) + t // 8 * (128 * u) + d % 16 * (8 * u) + d // 16 % u * 8 + t % 8
    return flat, k_at.reshape(-1), v_at.reshape(-1)


def _rows64(cache, scale, pages, which):
    flat, k_at, v_at = _untile(cache, scale, pages)
    H, bs, D = cache.shape[-3:]
    x = _bits(flat)[:, :, k_at if which == "k" else v_at].view(flat.dtype).double().reshape(-1, H, bs, D)
    if scale is not None:
        x = x * scale[pages].double()[..., None]
    return x.transpose(1, 2).reshape(-1, H, D)


def exact(case, seed):
    op = case["op"]
    if op in ("plan", "verify", "commit"):  # whole numbers and rows moved as they are
        return None
    s = prepare(case, seed)
    bs = s["block"]
    if op == "write":
        H, D = s["k"].shape[1:]

        def turned(x):
            x = x.double()
            if s["cos_sin"] is not None:
                cs = s["cos_sin"].double()[s["positions"].long()][:, None, :]
                h = cs.shape[-1] // 2
                z = torch.complex(x[..., :h], x[..., h:2 * h]) * torch.complex(cs[..., :h], cs[..., h:])
                x = torch.cat([z.real, z.imag, x[..., 2 * h:]], -1)
            return x

        q = turned(s["q"])
        if s["k_scale"] is not None:  # codes and the K scale go by values rounded to 16 bits: ties decide
            vs = torch.zeros(s["v_scale"].shape, dtype=torch.float64, device=DEV)
            vs[s["slots"] // bs, :, s["slots"] % bs] = s["v"].double().abs().amax(-1) / E4M3_MAX
            return q, None, None, None, vs
        out = []
        for which, x in (("k", turned(s["k"])), ("v", s["v"].double())):
            cache = s[which + "_cache"]
            rows = torch.zeros((cache.shape[0] * bs, H, D), dtype=torch.float64, device=DEV)
            rows[s["slots"]] = x
            rows = rows.reshape(-1, bs, H, D).transpose(1, 2).reshape(-1, H, bs * D)
            _, k_at, v_at = _untile(cache, None, slice(0, 0))
            tiled = torch.empty_like(rows)
            tiled[:, :, k_at if which == "k" else v_at] = rows
            out.append(tiled.reshape(cache.shape))
        return q, out[0], out[1], None, None
    H, D = s["k_cache"].shape[1], s["k_cache"].shape[3]
    q, G = s["q"].double(), s["q"].shape[1] // H
    o, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    start, kv = s["q_start"].tolist(), s["kv_lens"].tolist()
    for r, n in enumerate(kv):
        a, b = start[r], start[r + 1]
        pages = s["table"][r, :-(-n // bs)].long()
        k = _rows64(s["k_cache"], s["k_scale"], pages, "k")[:n]
        v = _rows64(s["v_cache"], s["v_scale"], pages, "v")[:n]
        c = n - (b - a)
        blind = torch.zeros((b - a, n), dtype=torch.bool, device=DEV)
        for i in range(b - a if s["mask"] is not None else 0):
            word = int(s["mask"][a + i]) & (2 ** 64 - 1)
            blind[i, c:] = torch.tensor([not (word >> j) & 1 for j in range(b - a)], device=DEV)
        if s["mask"] is None:
            blind[:, c:] = torch.ones((b - a, b - a), dtype=torch.bool, device=DEV).triu(1)
        for h in range(H):
            for u in range(h * G, (h + 1) * G):
                score = (q[a:b, u] @ k[:, h].t()) / math.sqrt(D)
                score.masked_fill_(blind, -math.inf)
                lse[a:b, u] = torch.logsumexp(score, 1)
                o[a:b, u] = torch.softmax(score, 1) @ v[:, h]
    return o, lse
