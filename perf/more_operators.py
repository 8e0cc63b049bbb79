"""Cases of a hybrid decoder's token mixers: what is measured, in plain torch and through the package.

A hybrid decoder has two kinds of layers between its linear layers.  Its attention layers normalise
every head of q and k, turn them by positions of one or several axes and write the cache
(kv_write_norm).  Its other layers keep a state of fixed size for each request: a short causal
convolution (short_conv) feeds the gated delta rule (delta_rule), for prompts, single tokens and drafted
trees; once a tree's branch is accepted, the states are taken along it (delta_commit).

With a state S [Dk, Dv] of each value head, log decay g and step size b, the delta rule is, token by token,
    S <- exp(g) S + k (b (v - exp(g) S^T k))^T,   out = scale S^T q;
a tree's token starts from its parent's state.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
MAX_NODES = 64
E4M3_MAX = 448.0
EPS = 1e-6


# --------------------------------------------------------------------------- cases
def listed():
    wide = dict(key_heads=16, group=3, dim_k=128, dim_v=128)
    return [
        # one user's drafted tree into one attention layer with wide heads: the call's latency
        dict(name="norm write one tree", op="write", tokens=33, kv_heads=4, group=6, head_dim=256, rot=64, axes=1,
             order="sections", gated=True, cache="bf16", block=16),
        # a token of each of 64 users into an 8-bit cache, positions of images among them
        dict(name="norm write token batch", op="write", tokens=64, kv_heads=8, group=4, head_dim=128, rot=128, axes=3,
             order="sections", gated=False, cache="e4m3", block=32),
        # an odd prompt with images, q beside its gate in the layer's rows
        dict(name="norm write prompt", op="write", tokens=8191, kv_heads=4, group=6, head_dim=256, rot=64, axes=3,
             order="interleaved", gated=True, cache="bf16", block=64),
        # a token of each of 64 users through one layer's convolution
        dict(name="conv token batch", op="conv", requests=64, nodes=1, ragged=False, tree=False, taps=4, **wide),
        # an odd prompt
        dict(name="conv prompt", op="conv", requests=1, nodes=8191, ragged=False, tree=False, taps=4, **wide),
        # one user, one token: latency
        dict(name="delta one token", op="delta", requests=1, nodes=1, ragged=False, tree=False, **wide),
        # a full server's decoding step: every request's state is read and written
        dict(name="delta token batch", op="delta", requests=64, nodes=1, ragged=False, tree=False, **wide),
        # a batch of drafted trees: the states are read only
        dict(name="delta trees", op="delta", requests=16, nodes=64, ragged=True, tree=True, **wide),
        # one odd prompt: the chain of its chunks
        dict(name="delta prompt", op="delta", requests=1, nodes=8191, ragged=False, tree=False, **wide),
        # prompts of very different lengths through a layer with narrow heads
        dict(name="delta prompt batch", op="delta", requests=24, nodes=1500, ragged=True, tree=False, key_heads=8,
             group=2, dim_k=64, dim_v=64),
        # one user's tree, one layer
        dict(name="delta commit one layer", op="commit", requests=1, nodes=17, layers=1, taps=4, **wide),
        # every such layer of a small batch in one call
        dict(name="delta commit all layers", op="commit", requests=4, nodes=16, layers=48, taps=4, **wide),
    ]


def _log(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["write", "conv", "delta", "delta", "delta", "commit"])
    if op == "write":
        dim = rng.choice([64, 128, 256])
        heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 8])
        return dict(op=op, tokens=_log(rng, 1, 8191 * 4 * 256 * 8 // (heads * (group + 2) * dim)), kv_heads=heads,
                    group=group, head_dim=dim, rot=rng.choice([0, dim // 4, dim // 2, dim]), axes=rng.choice([1, 2, 3]),
                    order=rng.choice(["sections", "interleaved"]), gated=rng.random() < 0.5,
                    cache=rng.choice(["bf16", "e4m3"]), block=rng.choice([16, 32, 64, 128]))
    heads = dict(key_heads=rng.choice([1, 2, 3, 4, 8, 16]), group=rng.choice([1, 2, 3, 4]), dim_k=rng.choice([64, 128]),
                 dim_v=rng.choice([32, 64, 128]))
    Hk, G, Dk, Dv = heads.values()
    if op == "commit":
        requests = _log(rng, 1, 32)
        most = 48 * 4 * 48 * 128 * 128 // (requests * Hk * G * Dk * Dv)
        return dict(op=op, requests=requests, nodes=_log(rng, 1, 64), layers=_log(rng, 1, max(1, min(48, most))),
                    taps=rng.choice([2, 3, 4]), **heads)
    tree = rng.random() < 0.4
    # tokens within the prompt's rows and states, requests within the token batch's states
    rows = 8191 * (32 * 128 + 48 * 128) // (2 * Hk * Dk + Hk * G * Dv)
    nodes = _log(rng, 1, min(64 if tree else 8191, rows))
    most = max(1, min(rows // nodes, 64 * 48 * 128 * 128 // (Hk * G * Dk * Dv)))
    return dict(op=op, requests=_log(rng, 1, min(256, most)), nodes=nodes, ragged=rng.random() < 0.6, tree=tree,
                **(dict(taps=rng.choice([2, 3, 4])) if op == "conv" else {}), **heads)


def _lengths(case):
    """New tokens of the requests, from the case alone: unevenly spread up to `nodes`, the longest first."""
    R, n = case["requests"], case["nodes"]
    if not case.get("ragged", True):
        return [n] * R
    return [int(1 + (n - 1) * (1.0 - (r * 0.6180339887498949) % 1.0)) for r in range(R)]


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _masks(rng, sizes):
    """Ancestor bits (the node's own among them) of every node of random trees, as int64."""
    out = []
    for n in sizes:
        m = []
        for i in range(n):
            p = i - 1 if rng.random() < 0.5 else int(rng.random() * i)
            m.append((m[p] if i else 0) | (1 << i))
        out += m
    return torch.from_numpy(np.array(out, dtype=np.uint64).view(np.int64)).to(DEV)


def _layer_rows(g, lead, case):
    """q, k, v as the convolution leaves them (columns of one tensor) and the gates' columns of a linear layer."""
    Hk, G, Dk, Dv = (case[n] for n in ("key_heads", "group", "dim_k", "dim_v"))
    y = _randn(g, lead + (2 * Hk * Dk + Hk * G * Dv,)) + 0.3
    y = y * torch.sigmoid(y)
    qk = y[..., :2 * Hk * Dk].unflatten(-1, (2 * Hk, Dk))
    y[..., :2 * Hk * Dk] = (qk * torch.rsqrt((qk * qk).sum(-1, keepdim=True) + EPS)).flatten(-2)
    y = y.to(torch.bfloat16)
    ab = _randn(g, lead + (2 * Hk * G,))
    return (y[..., :Hk * Dk].unflatten(-1, (Hk, Dk)), y[..., Hk * Dk:2 * Hk * Dk].unflatten(-1, (Hk, Dk)),
            y[..., 2 * Hk * Dk:].unflatten(-1, (Hk * G, Dv)), ab[..., :Hk * G], ab[..., Hk * G:])


def _gates(g, lead, heads):
    """a_log and dt_bias of a layer: decays from 0.2 to 0.999 a token."""
    rate = 1.0 + 15.0 * torch.rand(lead + (heads,), generator=g, device=DEV)
    dt = torch.exp(math.log(0.001) + math.log(100.0) * torch.rand(lead + (heads,), generator=g, device=DEV))
    return rate.log(), dt + torch.log(-torch.expm1(-dt))


def prepare(case, seed):
    g, rng, op = _gen(seed), np.random.default_rng(seed), case["op"]
    s = {"op": op}
    if op == "write":
        T, H, G, D, bs, rot = (case[k] for k in ("tokens", "kv_heads", "group", "head_dim", "block", "rot"))
        wide = D * (2 if case["gated"] else 1)
        qkv = 2.0 * _randn(g, (T, G * H * wide + 2 * H * D)) + 0.5
        qkv = qkv.to(torch.bfloat16)
        s["q"] = qkv[:, :G * H * wide].unflatten(1, (G * H, wide))[..., :D]
        s["k"] = qkv[:, G * H * wide:][:, :H * D].unflatten(1, (H, D))
        s["v"] = qkv[:, G * H * wide + H * D:].unflatten(1, (H, D))
        s["q_weight"], s["k_weight"] = (1.0 + 0.2 * _randn(g, (D,)) for _ in "qk")
        s["block"] = bs
        pages = -(-T // bs) + 3
        first = int(rng.integers(0, bs))
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(T, device=DEV) + first
        s["slots"] = order[at // bs] * bs + at % bs
        s["positions"], s["cos_sin"], s["axis_of"] = None, None, None
        if rot:
            h, A = rot // 2, case["axes"]
            base = at + int(rng.integers(0, 30000))
            patch = torch.arange(T, device=DEV) % 700 >= 100  # of every 700 tokens, 600 are an image of rows of 25
            cell = torch.arange(T, device=DEV) % 700 - 100
            steps = [-cell, cell // 25 - cell, cell % 25 - cell]
            pos = [torch.where(patch, base + steps[a], base) for a in range(A)]
            s["positions"] = (pos[0] if A == 1 else torch.stack(pos)).to(torch.int32).contiguous()
            pair = torch.arange(h, device=DEV)
            if A > 1:
                s["axis_of"] = (pair * A // h if case["order"] == "sections" else pair % A).to(torch.int32)
            f = 1e6 ** (-torch.arange(h, dtype=torch.float64, device=DEV) / h)
            a = torch.arange(131072 // 2, dtype=torch.float64, device=DEV)[:, None] * f
            s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        s["q_out"] = torch.empty((T, G * H, D), dtype=torch.bfloat16, device=DEV)
        kind = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
        for n in "kv":
            s[n + "_cache"] = torch.zeros((pages, H, bs, D), dtype=torch.uint8, device=DEV).to(kind)
            s[n + "_scale"] = None if case["cache"] == "bf16" else torch.zeros((pages, H, bs), device=DEV)
        return s
    Hk, G, Dk, Dv = (case[n] for n in ("key_heads", "group", "dim_k", "dim_v"))
    new = _lengths(case)
    R, T, C = len(new), sum(new), 2 * Hk * Dk + Hk * G * Dv
    s["widest"] = max(new)
    s["q_start"] = _ints([0] + np.cumsum(new).tolist())
    # one request in five has just begun: its state's slot still holds another's
    ctx = [0 if R > 1 and r % 5 == 4 else 1 + int(rng.integers(0, 4000)) for r in range(R)]
    s["kv_lens"] = _ints([c + n for c, n in zip(ctx, new)])
    s["state_slots"] = torch.randperm(R + 2, generator=g, device=DEV)[:R].to(torch.int32)
    s["mask"] = _masks(rng, new) if op == "commit" or case["tree"] else None
    lead = (case["layers"],) if op == "commit" else ()
    if op in ("conv", "commit"):
        s["x"] = _randn(g, lead + (T, C)).to(torch.bfloat16)
        s["conv_state"] = _randn(g, lead + (R + 2, case["taps"] - 1, C)).to(torch.bfloat16)
    if op == "conv":
        s["weight"], s["heads"] = 0.5 * _randn(g, (C, case["taps"])), (2 * Hk, Dk)
        s["out"] = torch.empty((T, C), dtype=torch.bfloat16, device=DEV)
        return s
    s["q"], s["k"], s["v"], s["a"], s["b"] = _layer_rows(g, lead + (T,), case)
    s["a_log"], s["dt_bias"] = _gates(g, lead, Hk * G)
    s["state"] = 0.2 * _randn(g, lead + (R + 2, Hk * G, Dk, Dv))
    if op == "delta":
        s["out"] = torch.empty((T, Hk * G, Dv), dtype=torch.bfloat16, device=DEV)
        return s
    path = np.full((R, MAX_NODES), -1, dtype=np.int32)  # accepted branches: from the deepest of a few nodes to the root
    count = np.zeros(R, dtype=np.int32)
    words, at = s["mask"].tolist(), 0
    for r, n in enumerate(new):
        tips = [words[at + int(i)] & (2 ** 64 - 1) for i in rng.integers(0, n, 4)]
        word = max(tips, key=lambda w: bin(w).count("1"))
        nodes = [i for i in range(n) if word >> i & 1]
        path[r, :len(nodes)], count[r] = nodes, len(nodes)
        at += n
    s["path"], s["accepted"] = torch.from_numpy(path).to(DEV), torch.from_numpy(count).to(DEV)
    return s


# --------------------------------------------------------------------------- plain forms: the cache
def _place(token):
    return token % 4 + token // 8 % 2 * 4 + token // 4 % 2 * 8


def _bits(cache):
    return cache.view(torch.int16 if cache.dtype == torch.bfloat16 else torch.uint8)


def _put_rows(which, cache, slots, block, rows):
    """rows [T, heads, D] into the cache's tiles of 16 tokens (matrix-operand order) at `slots`."""
    D, e, u = cache.shape[-1], *((8, 1) if cache.dtype == torch.bfloat16 else (16, 2))
    flat = _bits(cache).unflatten(-2, (-1, 16)).flatten(-2)             # [pages, heads, tiles, 16 D]
    b, i = slots // block, slots % block
    if which == "k":
        t = flat.unflatten(-1, (D // (4 * e), 4, 16, e))
        t[b, :, i // 16, :, :, _place(i % 16)] = _bits(rows).unflatten(-1, (-1, 4, e))
    else:
        t = flat.unflatten(-1, (D // (16 * u), 2, 16, u, 8))
        t[b, :, i // 16, :, i % 16 // 8, :, :, i % 8] = _bits(rows).unflatten(-1, (-1, u, 16)).transpose(-1, -2)


def _e4m3(x):
    top = x.float().abs().amax(-1)
    scale = top / torch.full_like(top, E4M3_MAX)  # a tensor: torch multiplies by a number's reciprocal instead
    code = torch.where(scale[..., None] > 0, x.float() / scale[..., None], 0.0)
    return code.to(torch.float8_e4m3fn), scale


def _normed(x, weight, s):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    if s["cos_sin"] is None:
        return x
    h = s["cos_sin"].shape[1] // 2
    pos = s["positions"].long()
    pair = torch.arange(h, device=x.device)
    at = pos[:, None].expand(-1, h) if s["axis_of"] is None else pos[s["axis_of"].long()].t()
    c, n = s["cos_sin"][at, pair][:, None, :], s["cos_sin"][at, pair + h][:, None, :]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat([a * c - b * n, b * c + a * n, x[..., 2 * h:]], -1)


def _write_plain(s):
    bs, slots = s["block"], s["slots"]
    s["q_out"].copy_(_normed(s["q"], s["q_weight"], s))
    k, v = _normed(s["k"], s["k_weight"], s), s["v"].contiguous()
    if s["k_scale"] is not None:
        k, ks = _e4m3(k)
        v, vs = _e4m3(v)
        s["k_scale"][slots // bs, :, slots % bs] = ks
        s["v_scale"][slots // bs, :, slots % bs] = vs
    _put_rows("k", s["k_cache"], slots, bs, k.to(s["k_cache"].dtype))
    _put_rows("v", s["v_cache"], slots, bs, v)
    return s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


# --------------------------------------------------------------------------- plain forms: convolution and delta rule
def _requests(s, T):
    """Of every token its request and number in it; of every request its length and whether it has just begun."""
    start = s["q_start"].long()
    t = torch.arange(T, device=start.device)
    r = torch.searchsorted(start[1:], t, right=True)
    n = start[1:] - start[:-1]
    return r, t - start[r], n, s["kv_lens"].long() - n <= 0


def _conv_plain(s):
    x, W, state = s["x"].float(), s["weight"], s["conv_state"]
    T, taps = x.shape[0], s["weight"].shape[1]
    r, i, n, fresh = _requests(s, T)
    old = torch.where(fresh[:, None, None], 0.0, state[s["state_slots"].long()].float())  # [R, taps - 1, C]
    y, at = x * W[:, -1], i
    for j in range(1, taps):  # the tap j tokens back: the chain's, or the tree's
        if s["mask"] is None:
            at = i - j
        else:
            below = s["mask"] & ((1 << at.clamp_min(0)) - 1)
            bit = (below[:, None] >> torch.arange(64, device=x.device)) & 1
            up = torch.where(bit > 0, torch.arange(64, device=x.device), -1).amax(1)
            at = torch.where(at > 0, torch.where(up >= 0, up, -1), at - 1)  # -1, -2, ..: the rows before the step
        row = torch.where((at >= 0)[:, None], x[(s["q_start"].long()[r] + at).clamp_min(0)],
                          old[r, (taps - 1 + at).clamp(0, taps - 2)])
        y = y + row * W[:, -1 - j]
    y = y * torch.sigmoid(y)
    heads, D = s["heads"]
    qk = y[:, :heads * D].unflatten(1, (heads, D))
    qk = qk * torch.rsqrt((qk * qk).sum(-1, keepdim=True) + EPS)
    s["out"].copy_(torch.cat([qk.flatten(1), y[:, heads * D:]], 1))
    if s["mask"] is None:
        back = n[:, None] - (taps - 1) + torch.arange(taps - 1, device=x.device)  # tokens of the new state
        new = torch.where((back >= 0)[..., None], x[(s["q_start"].long()[:-1, None] + back).clamp_min(0)],
                          torch.gather(old, 1, (back + taps - 1).clamp(0, taps - 2)[..., None].expand_as(old)))
        state[s["state_slots"].long()] = new.to(state.dtype)
    return s["out"], state


def _decay_and_step(a, b, a_log, dt_bias):
    return -torch.exp(a_log) * torch.nn.functional.softplus(a + dt_bias), torch.sigmoid(b)


def _chunks(q, k, v, g, b, state, word):
    """The delta rule over padded requests: q, k [R, N, Hk, Dk], v [R, N, Hv, Dv], g, b [R, N, Hv] (zeros where no
    token is), state [R, Hv, Dk, Dv]; word [R, N]: a tree's ancestors, or None.  Chunks of up to 64 tokens: with
    D the sum of log decays, U solves (I + A) U = b (V - exp(D) K S), A[i, j] = b_i exp(D_i - D_j) k_i k_j, j before i."""
    R, N, Hk, Dk = q.shape
    Hv, C = v.shape[2], min(N, MAX_NODES)
    q, k, v, g, b = (torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, -N % C)) for x in (q, k, v, g, b))
    cut = lambda x: x.unflatten(1, (-1, C)).transpose(2, 3)             # [R, chunks, heads, C, ..]
    q, k, v, g, b = (cut(x) for x in (q, k, v, g[..., None], b[..., None]))
    q, k = (x.repeat_interleave(Hv // Hk, 2) for x in (q, k))
    i = torch.arange(C, device=q.device)
    seen = (i[:, None] >= i).expand(R, 1, 1, C, C)
    if word is not None:
        seen = seen & ((word[:, None, None, :, None] >> i) & 1).bool()
    total = torch.matmul(seen.double(), g.double())                     # [R, chunks, Hv, C, 1]
    decay = torch.exp(torch.where(seen, total - total.transpose(3, 4), -math.inf).float())
    kt = k.transpose(3, 4).contiguous()
    A = torch.where(i[:, None] > i, b * decay * torch.matmul(k, kt), 0.0)
    inverse = torch.eye(C, device=q.device).expand_as(A).contiguous()
    for j in range(1, C):
        inverse[..., j, :j] = -torch.matmul(A[..., j:j + 1, :j], inverse[..., :j, :j].contiguous())[..., 0, :]
    P = decay * torch.matmul(q, kt)
    grown = torch.exp(total.float())
    last = total[..., -1:, :]
    left = torch.exp((last - total).float()).transpose(3, 4) * kt
    out = []
    for c in range(q.shape[1]):
        u = torch.matmul(inverse[:, c], b[:, c] * (v[:, c] - grown[:, c] * torch.matmul(k[:, c], state)))
        out.append(grown[:, c] * torch.matmul(q[:, c], state) + torch.matmul(P[:, c], u))
        state = torch.exp(last[:, c].float()) * state + torch.matmul(left[:, c], u)
    return torch.stack(out, 1).transpose(2, 3).flatten(1, 2), state


def _padded(x, s, n):
    at = (s["q_start"].long()[:-1, None] + torch.arange(n, device=x.device)).clamp_max(x.shape[0] - 1)
    there = torch.arange(n, device=x.device) < (s["q_start"][1:] - s["q_start"][:-1])[:, None]
    return torch.where(there.reshape(there.shape + (1,) * (x.dim() - 1)), x[at].float(), 0.0)


def _delta_plain(s):
    r, i, _, fresh = _requests(s, s["q"].shape[0])
    g, b = _decay_and_step(s["a"], s["b"], s["a_log"], s["dt_bias"])
    q, k, v, g, b = (_padded(x, s, s["widest"]) for x in (s["q"], s["k"], s["v"], g, b))
    word = None
    if s["mask"] is not None:
        at = s["q_start"].long()[:-1, None] + torch.arange(s["widest"], device=q.device)
        word = s["mask"][at.clamp_max(s["mask"].numel() - 1)]
    slots = s["state_slots"].long()
    state = torch.where(fresh[:, None, None, None], 0.0, s["state"][slots])
    out, state = _chunks(q, k, v, g, b, state, word)
    s["out"].copy_(out[r, i] * q.shape[-1] ** -0.5)
    if s["mask"] is None:
        s["state"][slots] = state
    return s["out"], s["state"]


def _commit_plain(s):
    path, first = s["path"].long(), s["q_start"].long()[:-1, None]
    *_, fresh = _requests(s, s["k"].shape[1])
    L, (R, n) = s["k"].shape[0], path.shape
    go = torch.arange(n, device=path.device) < s["accepted"][:, None]
    at = (first + path).clamp(0, s["k"].shape[1] - 1)
    g, b = _decay_and_step(s["a"], s["b"], s["a_log"][:, None], s["dt_bias"][:, None])
    rows = lambda x: torch.where(go.reshape(R, n, *(1,) * (x.dim() - 2)), x[:, at].float(), 0.0).flatten(0, 1)
    slots = s["state_slots"].long()
    state = torch.where(fresh[:, None, None, None], 0.0, s["state"][:, slots])
    _, state = _chunks(rows(s["k"]), rows(s["k"]), rows(s["v"]), rows(g), rows(b), state.flatten(0, 1), None)
    s["state"][:, slots] = state.unflatten(0, (L, R))
    taps = s["conv_state"].shape[2]
    old = torch.where(fresh[:, None, None], 0.0, s["conv_state"][:, slots].float())
    back = s["accepted"].long()[:, None] - taps + torch.arange(taps, device=path.device)
    row = (first + torch.gather(path, 1, back.clamp_min(0))).clamp(0, s["x"].shape[1] - 1)
    before = old[:, torch.arange(R, device=path.device)[:, None], (back + taps).clamp_max(taps - 1)]
    s["conv_state"][:, slots] = torch.where((back >= 0)[..., None], s["x"][:, row].float(), before).to(torch.bfloat16)
    return s["state"], s["conv_state"]


def run(s):
    op = s["op"]
    if not own:
        return {"write": _write_plain, "conv": _conv_plain, "delta": _delta_plain, "commit": _commit_plain}[op](s)
    import quantized_gemv_gemm_amd as tl
    if op == "write":
        tl.kv_write_norm(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"],
                         v_scale=s["v_scale"], q=s["q"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                         positions=s["positions"], cos_sin=s["cos_sin"], axis_of=s["axis_of"], q_out=s["q_out"])
        return s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if op == "conv":
        tl.short_conv(s["x"], s["weight"], s["q_start"], s["kv_lens"], s["state_slots"], s["conv_state"],
                      tree_mask=s["mask"], norm_heads=s["heads"][0], norm_dim=s["heads"][1], eps=EPS, out=s["out"])
        return s["out"], s["conv_state"]
    if op == "delta":
        tl.delta_rule(s["q"], s["k"], s["v"], s["a"], s["b"], s["q_start"], s["kv_lens"], s["state_slots"], s["state"],
                      a_log=s["a_log"], dt_bias=s["dt_bias"], tree_mask=s["mask"], max_nodes=s["widest"], out=s["out"])
        return s["out"], s["state"]
    tl.delta_commit(s["accepted"], s["path"], s["q_start"], s["kv_lens"], s["state_slots"], s["k"], s["v"], s["a"], s["b"],
                    s["state"], a_log=s["a_log"], dt_bias=s["dt_bias"], x=s["x"], conv_state=s["conv_state"])
    return s["state"], s["conv_state"]


# --------------------------------------------------------------------------- work and the exact values
def work(case):
    op = case["op"]
    if op == "write":
        T, H, G, D = (case[n] for n in ("tokens", "kv_heads", "group", "head_dim"))
        row = H * (D * 2 if case["cache"] == "bf16" else D + 4)
        return {"bytes": T * (2 * D * H * (G + 2) + 2 * D * H * G + 2 * row + 8 + 4 * case["rot"] + 4 * case["axes"]),
                "flops": T * H * ((G + 1) * (4 * D + 3 * case["rot"]) + (0 if case["cache"] == "bf16" else 2 * D))}
    Hk, G, Dk, Dv = (case[n] for n in ("key_heads", "group", "dim_k", "dim_v"))
    new = _lengths(case)
    R, T, C = len(new), sum(new), 2 * Hk * Dk + Hk * G * Dv
    state, kv = 4 * Hk * G * Dk * Dv, 2 * Hk * Dk + 2 * Hk * G * Dv + 8 * Hk * G
    if op == "conv":
        kept = 2 * R * (case["taps"] - 1) * C
        return {"bytes": 4 * T * C + kept * (1 if case["tree"] else 2) + 4 * C * case["taps"] + 8 * T * case["tree"],
                "flops": T * C * (2 * case["taps"] + 6)}
    if op == "delta":
        return {"bytes": T * (kv + 2 * Hk * Dk + 2 * Hk * G * Dv + 8 * case["tree"]) + R * state * (1 if case["tree"] else 2),
                "flops": 6 * T * Hk * G * Dk * Dv}
    taken = sum(min(n, 1 + n.bit_length()) for n in new)  # about the depth of a random tree
    return {"bytes": case["layers"] * (2 * R * state + taken * kv + R * (case["taps"] - 1) * C * 4),
            "flops": case["layers"] * 4 * taken * Hk * G * Dk * Dv}


def _parent(word, i):
    """A tree node's parent from its word of ancestors; -1 for the root."""
    return (int(word) & ((1 << i) - 1)).bit_length() - 1


def _step64(S, k, v, a, b, a_log, dt_bias):
    """One token of a request: states [.., Hv, Dk, Dv] in 64 bits after it."""
    z = (a + dt_bias).double()
    g = -a_log.double().exp() * (z.clamp_min(0) + torch.log1p(torch.exp(-z.abs())))
    S = S * g.exp()[..., None, None]
    k = k.double().repeat_interleave(S.shape[-3] // k.shape[-2], -2)
    miss = v.double() - (S * k[..., None]).sum(-2)
    return S + k[..., None] * (miss / (1 + torch.exp(-b.double()))[..., None])[..., None, :]


def exact(case, seed):
    op, s = case["op"], prepare(case, seed)
    if op == "write":
        H, D = s["k"].shape[1:]

        def turned(x, weight):
            x = x.double()
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.double()
            if s["cos_sin"] is not None:
                h = s["cos_sin"].shape[1] // 2
                pos = s["positions"].reshape(-1, x.shape[0]).long()
                axis = torch.zeros(h, dtype=torch.long, device=DEV) if s["axis_of"] is None else s["axis_of"].long()
                cols = [torch.complex(s["cos_sin"][pos[axis[j]], j].double(), s["cos_sin"][pos[axis[j]], j + h].double())
                        for j in range(h)]
                z = torch.complex(x[..., :h], x[..., h:2 * h]) * torch.stack(cols, 1)[:, None, :]
                x = torch.cat([z.real, z.imag, x[..., 2 * h:]], -1)
            return x

        q, k, v = turned(s["q"], s["q_weight"]), turned(s["k"], s["k_weight"]), s["v"].double()
        if s["k_scale"] is not None:  # codes go by borders between values: ties decide
            scales = []
            for x in (k, v):
                scales.append(torch.zeros(s["k_scale"].shape, dtype=torch.float64, device=DEV))
                scales[-1][s["slots"] // s["block"], :, s["slots"] % s["block"]] = x.abs().amax(-1) / E4M3_MAX
            return q, None, None, *scales
        out, bs = [], s["block"]
        t, d = torch.meshgrid(torch.arange(bs, device=DEV), torch.arange(D, device=DEV), indexing="ij")
        tile, m = t // 16 * (16 * D), t % 16
        k_at = tile + d // 32 * 512 + d % 32 // 8 * 128 + ((m & 3) | (m & 8) >> 1 | (m & 4) << 1) * 8 + d % 8
        v_at = tile + d // 16 * 256 + m // 8 * 128 + d % 16 * 8 + m % 8
        for at, x in ((k_at, k), (v_at, v)):
            cache = s["k_cache"]
            rows = torch.zeros((cache.shape[0] * bs, H, D), dtype=torch.float64, device=DEV)
            rows[s["slots"]] = x
            tiled = torch.empty((cache.shape[0], H, bs * D), dtype=torch.float64, device=DEV)
            tiled[:, :, at.reshape(-1)] = rows.reshape(-1, bs, H, D).transpose(1, 2).reshape(-1, H, bs * D)
            out.append(tiled.reshape(cache.shape))
        return q, out[0], out[1], None, None
    start, kv, slots = s["q_start"].tolist(), s["kv_lens"].tolist(), s["state_slots"].tolist()
    new = [b - a for a, b in zip(start, start[1:])]
    words = None if s["mask"] is None else [w & (2 ** 64 - 1) for w in s["mask"].tolist()]
    if op == "conv":
        if words is not None and start[-1] > 20000:
            return None
        taps, state = s["weight"].shape[1], s["conv_state"].double()
        out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
        w = s["weight"].double()
        for r, n in enumerate(new):
            x, old = s["x"][start[r]:start[r + 1]].double(), state[slots[r]].clone()
            if kv[r] <= n:
                old.zero_()
            rows = torch.cat([old, x])
            at = []
            for i in range(n):
                line = [i]
                for _ in range(1, taps):
                    j = line[-1]
                    line.append(_parent(words[start[r] + i], j) if words is not None and j > 0 else j - 1)
                at.append(line)
            at = torch.tensor(at, device=DEV) + taps - 1
            y = sum(rows[at[:, j]] * w[:, taps - 1 - j] for j in range(taps))
            out[start[r]:start[r + 1]] = y / (1 + torch.exp(-y))
            if words is None:
                state[slots[r]] = rows[-(taps - 1):]
        heads, D = s["heads"]
        qk = out[:, :heads * D].unflatten(1, (heads, D))
        out[:, :heads * D] = (qk / torch.sqrt((qk * qk).sum(-1, keepdim=True) + EPS)).flatten(1)
        return out, state if words is None else None
    state = s["state"].double()
    if op == "commit":
        for r in range(len(new)):
            S = state[:, slots[r]] * (1.0 if kv[r] > new[r] else 0.0)
            for i in s["path"][r, :int(s["accepted"][r])].tolist():
                t = start[r] + i
                S = _step64(S, s["k"][:, t], s["v"][:, t], s["a"][:, t], s["b"][:, t], s["a_log"], s["dt_bias"])
            state[:, slots[r]] = S
        return state, None
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
    G = s["v"].shape[1] // s["k"].shape[1]
    gates = (s["a_log"], s["dt_bias"])
    # requests side by side, the longest first; a tree's nodes keep their states for their children
    order = sorted(range(len(new)), key=lambda r: -new[r])
    S = torch.stack([state[slots[r]] * (1.0 if kv[r] > new[r] else 0.0) for r in order])
    kept = [] if words is not None else None
    for i in range(max(new)):
        on = [r for r in order if new[r] > i]
        t = torch.tensor([start[r] + i for r in on], device=DEV)
        if words is not None:
            if i == 0:
                root = S
            up = [_parent(words[start[r] + i], i) for r in on]
            S = torch.stack([root[j] if p < 0 else kept[p][j] for j, p in enumerate(up)])
        done = _step64(S[:len(on)], s["k"][t], s["v"][t], s["a"][t], s["b"][t], *gates)
        out[t] = (done * s["q"][t].double().repeat_interleave(G, 1)[..., None]).sum(-2) / math.sqrt(s["q"].shape[-1])
        if words is not None:
            kept.append(done)
        else:
            S[:len(on)] = done
    if words is not None:
        return out, None
    for j, r in enumerate(order):
        state[slots[r]] = S[j]
    return out, state
