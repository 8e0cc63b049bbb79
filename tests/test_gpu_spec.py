"""Speculative-decoding operators on the GPU against their plain definitions in 64 bits
(oracle/speculative.py).  Whole numbers, moved rows and 8-bit codes are exact; computed
values stay within bounds counted from the roundings the kernels make."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle.speculative as ref
from gpu_common import announce, dev, to_dev

pytestmark = pytest.mark.gpu

BF16_HALF = 2.0 ** -8      # half a step of bfloat16, relative
F32_HALF = 2.0 ** -24


@pytest.fixture(scope="module")
def tl():
    import quantized_gemv_gemm_amd as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def torch():
    import torch
    return torch


def raw(t):
    """Raw element bits as numpy."""
    import torch
    kind = {torch.bfloat16: torch.int16, torch.float8_e4m3fn: torch.uint8}[t.dtype]
    return t.view(kind).cpu().numpy()


def values(bits):
    if bits.dtype == np.uint8:
        return ref.e4m3_value(bits)
    return (bits.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def randn_bf16(rng, shape, scale=1.0):
    return ref.bf16(scale * rng.standard_normal(shape))


def bf16_dev(x, d):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(torch.bfloat16).to(d)


# --------------------------------------------------------------------------- step_plan
def run_plan(tl, torch, ctx, new, owned, table, free, head, T, block, parents):
    d = dev()
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=d)
    tab = i32(table)
    got = tl.step_plan(i32(ctx), i32(new), i32(owned), tab, i32(free), i32([head]), T, block,
                       parents=None if parents is None else i32(parents))
    torch.cuda.synchronize()
    want = ref.step_plan(np.array(ctx), np.array(new), np.array(owned), np.array(table).reshape(len(ctx), -1),
                         np.array(free), head, T, block, parents)
    q, kv, slots, pos, mask, owned_w, head_w, table_w = want
    for name, g, w in (("q_start", got[0], q), ("kv_lens", got[1], kv), ("slots", got[2], slots), ("positions", got[3], pos),
                       ("owned", got[5], owned_w), ("head", got[6], [head_w]), ("table", tab, table_w)):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
    if parents is None:
        assert got[4] is None
    else:
        np.testing.assert_array_equal(got[4].cpu().numpy().view(np.uint64), mask, err_msg="tree_mask")


@pytest.mark.parametrize("R,block,tree,short", [(1, 16, True, 0), (1, 16, False, 0), (3, 32, True, 2), (70, 16, True, 5),
                                                (257, 64, False, 9), (600, 16, True, 0), (4096, 128, True, 40)])
def test_step_plan(tl, torch, R, block, tree, short):
    announce(f"step_plan R={R} block={block} tree={tree} short={short}")
    rng = np.random.default_rng(R + block)
    new = rng.choice([0, 1, 2, 17, 33, 63, 64, 65, 130], R)
    ctx = rng.integers(0, 300, R)
    ctx[rng.random(R) < 0.2] = 0
    owned = -(-ctx // block) + rng.integers(0, 2, R)          # pages left over from rejected nodes
    width = int(max(-(-(ctx + new) // block).max(), owned.max())) - (1 if R > 2 else 0)  # one too few for the longest
    owned = np.minimum(owned, width)
    table = rng.permutation(R * width + 5)[:R * width].reshape(R, width)
    need = np.maximum(0, -(-(ctx + new) // block) - owned).sum()
    free = rng.permutation(max(int(need) + 3 - short, 1)) + R * width
    T = int(new.sum()) + (7 if R % 2 else 0)
    parents = None
    if tree:
        parents = np.concatenate([np.where(rng.random(n) < 0.1, rng.integers(-3, 70, n),
                                           (rng.random(n) * np.arange(n)).astype(int)) for n in new] + [np.zeros(T - new.sum(), int)])
    run_plan(tl, torch, ctx, new, owned, table, free, 0, T, block, parents)


def test_step_plan_edges(tl, torch):
    announce("step_plan edges: nothing to do, no free page, tokens beyond the capacity, negative numbers")
    run_plan(tl, torch, [0, 5], [0, 0], [0, 1], [[1, 2], [3, 4]], [7], 0, 0, 16, None)
    run_plan(tl, torch, [16], [1], [1], [[3, 9]], [7], 1, 1, 16, [-1])       # head past the list
    run_plan(tl, torch, [16], [1], [1], [[3, 9]], [7], -1, 1, 16, [-1])
    run_plan(tl, torch, [4, 4], [40, 40], [0, 0], [[0] * 4] * 2, list(range(10)), 2, 50, 16, list(range(-1, 49)))
    run_plan(tl, torch, [-4, 3], [-2, 2], [-1, 0], [[0] * 4] * 2, list(range(10)), 0, 2, 16, None)


# --------------------------------------------------------------------------- kv_write
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,H,Hq,D,rot,block,first", [
    (1, 1, 1, 64, 0, 16, 0), (1, 4, 24, 256, 64, 16, 5), (7, 2, 6, 128, 128, 16, 3), (16, 1, 8, 128, 64, 32, 0),
    (33, 3, 3, 64, 32, 16, 15), (100, 2, 5, 256, 256, 64, 9), (50, 8, 0, 128, 16, 128, 120), (257, 1, 2, 64, 64, 32, 30)])
def test_kv_write(tl, torch, T, H, Hq, D, rot, block, first, e4m3):
    announce(f"kv_write T={T} H={H} Hq={Hq} D={D} rot={rot} block={block} first={first} e4m3={e4m3}")
    d, rng = dev(), np.random.default_rng(T * 7 + D + rot)
    x = randn_bf16(rng, (T, (Hq + 2 * H) * D + 8), 2.0)                # rows of a wider qkv output
    x[rng.random(T) < 0.1] = 0.0                                       # rows of zeros
    xd = bf16_dev(x, d)
    part = lambda a, n: (x[:, a:a + n * D].reshape(T, n, D), xd[:, a:a + n * D].unflatten(1, (n, D)))
    (k, kd), (v, vd) = part(Hq * D, H), part((Hq + H) * D, H)
    q, qd = part(0, Hq) if Hq else (None, None)
    pages = -(-(T + first) // block) + 2
    order, at = rng.permutation(pages), np.arange(T) + first
    slots = order[at // block] * block + at % block
    skip = rng.random(T) < 0.1
    slots = np.where(skip, rng.choice([-1, -5, pages * block, 1 << 40], T), slots).astype(np.int64)
    if T > 40:                                                         # a tree's nodes in between: slots out of order
        slots[20:30] = slots[20:30][::-1].copy()
    positions = rng.integers(-2, 5000, T).astype(np.int32)
    cs = None
    if rot:
        a = rng.uniform(0, 6.28, (4096, rot // 2))
        cs = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    kc, vc, ks, vs = tl.kv_cache(pages, H, block, D, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device=d)
    fill = 0x5A
    kc.view(torch.uint8).fill_(fill)
    vc.view(torch.uint8).fill_(fill)
    if e4m3:
        ks.fill_(-3.0)
        vs.fill_(-3.0)
    got = tl.kv_write(kd, vd, to_dev(slots, d), kc, vc, k_scale=ks, v_scale=vs, q=qd,
                      positions=to_dev(positions, d) if rot else None, cos_sin=None if cs is None else to_dev(cs, d))
    torch.cuda.synchronize()

    def turned(a):
        """The formula in f32, rounded at each step, and in 64 bits."""
        if not rot:
            return a, a
        h = rot // 2
        f = a.astype(np.float32)
        row = cs[np.clip(positions, 0, 4095)][:, None, :]
        c, s = row[..., :h], row[..., h:]
        lo, hi = f[..., :h], f[..., h:rot]
        out = f.copy()
        out[..., :h], out[..., h:rot] = lo * c - hi * s, hi * c + lo * s
        return ref.bf16(out), ref.rotate(a, cs, positions)

    def near(got64, exact64, a):
        h = rot // 2
        size = np.abs(a)
        if rot:
            both = size[..., :h] + size[..., h:rot]
            size = np.concatenate([both, both, size[..., rot:]], -1)
        assert (np.abs(got64 - exact64) <= BF16_HALF * np.abs(exact64) + 4 * F32_HALF * size).all()
    if Hq:
        want, exact = turned(q)
        g = values(raw(got))
        np.testing.assert_array_equal(g, want)
        near(g, exact, q)
    else:
        assert got is None
    want_k, exact_k = turned(k)
    near(want_k, exact_k, k)
    es = 1 if e4m3 else 2
    rk, rv = raw(kc), raw(vc)
    wk, wv = np.full_like(rk, fill if e4m3 else 0x5A5A), np.full_like(rv, fill if e4m3 else 0x5A5A)
    wks, wvs = np.full((pages, H, block), -3.0, np.float32), np.full((pages, H, block), -3.0, np.float32)

    def codes(a):
        scale = (np.abs(a).max(-1).astype(np.float32) / np.float32(448))
        with np.errstate(invalid="ignore", divide="ignore"):
            y = np.where(scale[..., None] > 0, a.astype(np.float32) / scale[..., None], np.float32(0))
        c = ref.e4m3_code(y)
        # against the exact value: half a step of 3 mantissa bits, or of the smallest numbers' spacing
        assert (np.abs(ref.e4m3_value(c) * scale[..., None].astype(np.float64) - a)
                <= (2.0 ** -4 + 2 * F32_HALF) * np.abs(a) + 2.0 ** -10 * scale[..., None].astype(np.float64)).all()
        return c, scale
    for cache, scales, a, which in ((wk, wks, want_k, "k"), (wv, wvs, v, "v")):
        bits, scale = codes(a) if e4m3 else ((a.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16).view(np.int16), None)
        at = ref.offsets(which, es, block, D)
        for t in range(T):
            if 0 <= slots[t] < pages * block:
                pg, tok = slots[t] // block, slots[t] % block
                for hh in range(H):
                    cache[pg, hh].reshape(-1)[at[tok]] = bits[t, hh]
                    if e4m3:
                        scales[pg, hh, tok] = scale[t, hh]
    np.testing.assert_array_equal(rk, wk)
    np.testing.assert_array_equal(rv, wv)
    if e4m3:
        np.testing.assert_array_equal(ks.cpu().numpy(), wks)
        np.testing.assert_array_equal(vs.cpu().numpy(), wvs)


# --------------------------------------------------------------------------- tree_attention
class Case:
    """Requests [(new, context)], a filled cache and everything a call needs."""

    def __init__(self, tl, requests, H, G, D, e4m3, block, tree=True, seed=0, pages=None, qscale=2.0):
        import torch
        self.tl, self.d, rng = tl, dev(), np.random.default_rng(seed)
        self.rng, self.H, self.G, self.D, self.block, self.e4m3 = rng, H, G, D, block, e4m3
        self.new = [n for n, _ in requests]
        self.kv = np.array([n + c for n, c in requests], dtype=np.int32)
        self.q_start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.T = int(self.q_start[-1])
        need = [-(-int(n) // block) for n in self.kv]
        self.pages = pages or sum(need) + 3
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(requests), max(max(need), 1)), 1 << 30, dtype=np.int32)  # entries past the end: not pages
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
        shape = (self.pages, H, block, D)
        es = 1 if e4m3 else 2
        self.es = es
        if e4m3:
            bits = rng.integers(0, 0x70, shape, dtype=np.uint8) | (rng.integers(0, 2, shape, dtype=np.uint8) << 7)
            self.kbits, self.vbits = bits, rng.permutation(bits.reshape(-1)).reshape(shape)
            self.ks = np.exp(0.3 * rng.standard_normal(shape[:3])).astype(np.float32) * np.float32(0.02)
            self.vs = np.exp(0.3 * rng.standard_normal(shape[:3])).astype(np.float32) * np.float32(0.02)
        else:
            f = lambda: (ref.bf16(rng.standard_normal(shape)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16).view(np.int16)
            self.kbits, self.vbits, self.ks, self.vs = f(), f(), None, None
        self.q = randn_bf16(rng, (self.T, H * G, D), qscale)
        self.mask = None
        if tree:
            words = []
            for n in self.new:
                m = []
                for i in range(n):
                    p = int(rng.integers(-1, i)) if i else -1
                    m.append(((m[p] if p >= 0 else 0) | 1 << i) if n <= 64 else 0)
                words += m
            self.mask = np.array(words, dtype=np.uint64)
        self.scale = None

    def call(self, max_nodes="known", q=None, **more):
        import torch
        d = self.d
        kind = torch.float8_e4m3fn if self.e4m3 else torch.bfloat16
        dv = lambda a: None if a is None else to_dev(a, d)
        self.out = torch.full((self.T, self.H * self.G, self.D), 777.0, dtype=torch.bfloat16, device=d)
        self.lse = torch.full((self.T, self.H * self.G), 777.0, dtype=torch.float32, device=d)
        most = max(self.new + [1]) if max_nodes == "known" else max_nodes
        self.args = dict(
            q=bf16_dev(self.q, d) if q is None else q, k_cache=dv(self.kbits).view(kind), v_cache=dv(self.vbits).view(kind),
            block_table=dv(self.table), q_start=dv(self.q_start), kv_lens=dv(self.kv),
            tree_mask=None if self.mask is None else dv(self.mask.view(np.int64)), k_scale=dv(self.ks), v_scale=dv(self.vs),
            scale=self.scale, max_nodes=most, out=self.out, lse=self.lse)
        self.args.update(more)
        announce(f"tree_attention requests={list(zip(self.new, (self.kv - np.diff(self.q_start)).tolist()))[:6]} H={self.H} G={self.G} "
                 f"D={self.D} e4m3={self.e4m3} block={self.block} max_nodes={most} mask={self.mask is not None}")
        self.tl.tree_attention(**self.args)
        torch.cuda.synchronize()
        return self

    def check(self, only=None):
        got, lse = values(raw(self.out)), self.lse.cpu().numpy().astype(np.float64)
        scale = self.D ** -0.5 if self.scale is None else self.scale
        for r in range(len(self.new)) if only is None else only:
            a, b, n = int(self.q_start[r]), int(self.q_start[r + 1]), int(self.kv[r])
            if b == a:
                continue
            ok = ref.there(self.table[r], self.pages, self.block, n)
            raws = [ref.rows(c, w, self.block, self.D, self.es, self.table[r], n) for c, w in ((self.kbits, "k"), (self.vbits, "v"))]
            k, v = (values(x) for x in raws)
            if self.e4m3:
                pos = np.arange(n)
                page = np.clip(self.table[r][pos // self.block], 0, self.pages - 1)
                k = k * self.ks[page, :, pos % self.block].astype(np.float64)[..., None]
                v = v * self.vs[page, :, pos % self.block].astype(np.float64)[..., None]
            v = np.where(ok[:, None, None], v, 0.0)
            k = np.where(ok[:, None, None], k, 0.0)
            mask = None if self.mask is None else self.mask[a:b]
            for h in range(self.H):
                rows = slice(h * self.G, (h + 1) * self.G)
                q = self.q[a:b, rows]
                want, wl = ref.attention(q, k[:, h], v[:, h], ok, b - a, mask, scale)
                self._near(got[a:b, rows], lse[a:b, rows], want, wl, q, k[:, h], v[:, h], ok, mask, scale, n)
        return self

    def _near(self, got, lse, want, wl, q, k, v, ok, mask, scale, n):
        fin = np.isfinite(k).all(-1) & ok
        # scores: products of 16-bit numbers are exact in f32, their sum of D terms and the scales' products
        # are off by up to (D + 8) half steps of the sum of magnitudes; the exponent by a few of |s| + |max|
        size = scale * (np.abs(q) @ np.abs(k[fin]).T).max(-1) if fin.any() else np.zeros(q.shape[:2])
        es = (self.D + 8) * F32_HALF * size + 16 * F32_HALF * (1 + size)
        keys = max(n, 1)
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(lse), empty)
        good = np.isfinite(wl)
        assert (np.abs(lse - wl)[good] <= (es + keys * F32_HALF + 8 * F32_HALF * (1 + np.abs(wl)))[good]).all()
        assert (got[empty] == 0).all()
        # sum of w |v| over the keys a row sees, from the same definition
        absolute, _ = ref.attention(q, k, np.abs(v), ok, len(q), mask, scale)
        bad = ~np.isfinite(want)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[bad & ~np.isnan(want)], want[bad & ~np.isnan(want)])
        # each probability (with its scale) is rounded once to bf16, the result once; f32 sums over the keys
        tol = 1.01 * ((BF16_HALF + 2 * es[..., None] + 2 * keys * F32_HALF) * absolute + BF16_HALF * np.abs(want)) + 1e-37
        assert (np.abs(got - want)[~bad] <= tol[~bad]).all(), np.nanmax(np.where(bad, 0, np.abs(got - want) / tol))


LENS = [(1, 0), (1, 1), (1, 14), (1, 15), (1, 16), (1, 31), (1, 32), (1, 63), (1, 126), (1, 127), (1, 128), (1, 500)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_single_tokens(tl, D, e4m3):
    Case(tl, LENS, 2, 3, D, e4m3, 16, seed=D).call().check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,G,nodes", [(64, 1, 16), (64, 4, 8), (64, 8, 64), (128, 1, 1), (128, 3, 5), (128, 5, 33),
                                       (128, 8, 4), (128, 64, 3), (256, 1, 9), (256, 6, 5), (256, 2, 64), (256, 7, 17)])
def test_attention_trees(tl, D, G, nodes, e4m3):
    """Every form (rows of a cache head: up to 16, up to 32, more), trees of other sizes beside the largest."""
    reqs = [(nodes, 100), (max(1, nodes // 2), 0), (nodes, 17), (1, 333), (0, 40), (max(1, nodes - 1), 31)]
    Case(tl, reqs, 2, G, D, e4m3, 32, seed=nodes + G).call().check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_long_split_over_workgroups(tl, D, e4m3):
    """Few heads and long caches: every item falls to many workgroups, whose sums are joined."""
    Case(tl, [(3, 9000), (9, 2000)], 1, 4, D, e4m3, 64, seed=1).call().check()
    Case(tl, [(40, 5000), (64, 700)], 1, 2, D, e4m3, 64, seed=2).call().check()
    Case(tl, [(1, 20001)], 1, 1, D, e4m3, 128, seed=3).call().check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 4), (256, 3)])
def test_attention_chains(tl, D, G, e4m3):
    """Without masks, and prompt chunks above 64 tokens with and without them."""
    Case(tl, [(1, 5), (2, 30), (64, 10), (7, 0)], 2, G, D, e4m3, 16, tree=False, seed=4).call().check()
    Case(tl, [(65, 0), (100, 37), (3, 50), (200, 0)], 1, G, D, e4m3, 16, tree=False, seed=5).call().check()
    Case(tl, [(130, 11), (10, 64), (66, 3)], 1, G, D, e4m3, 32, tree=True, seed=6).call().check()


def test_attention_many_requests(tl):
    """More requests than threads of a workgroup, most of them short, some empty."""
    rng = np.random.default_rng(8)
    reqs = [(int(n), int(c)) for n, c in zip(rng.choice([0, 1, 2, 5], 300), rng.choice([0, 1, 20, 60], 300))]
    Case(tl, reqs, 1, 2, 64, False, 16, seed=8).call().check()


@pytest.mark.parametrize("hint", [1, 3, 20, 1000])
def test_attention_hint_only_chooses(tl, hint):
    """max_nodes below and above the real number."""
    Case(tl, [(12, 40), (70, 3), (1, 200)], 1, 3, 128, False, 16, seed=9).call(max_nodes=hint).check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_rows_that_see_nothing(tl, e4m3):
    c = Case(tl, [(8, 0), (5, 40), (4, 0), (70, 0)], 2, 2, 128, e4m3, 16, seed=10)
    c.mask[:8] = [0, 1, 0, 9, 0, 32, 0, 255]
    c.mask[8:13] = 0                                   # sees the context alone
    c.kv[2] = 0                                        # not served
    c.kv[3] = 50                                       # fewer keys than tokens: the first 20 see none
    c.call().check()
    assert (values(raw(c.out))[13:17] == 0).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_bad_pages(tl, e4m3):
    """Pages outside the cache in the middle, at the end and everywhere: their tokens are not there."""
    c = Case(tl, [(4, 200), (4, 100), (2, 60)], 2, 2, 64, e4m3, 16, seed=11)
    c.table[0, 3], c.table[0, 7], c.table[1, 0] = -1, c.pages, 1 << 30
    c.table[2, :] = -7
    c.call().check()
    assert (values(raw(c.out))[8:] == 0).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,G,n", [(128, 2, 6), (64, 4, 20), (256, 3, 12)])
def test_attention_not_finite_where_masked(tl, D, G, n, e4m3):
    """NaN and infinities in every token past a request's end, and in nodes that some rows see and others do not."""
    c = Case(tl, [(n, 37), (n, 0)], 2, G, D, e4m3, 16, seed=12)
    inf = 0x7F if e4m3 else 0x7F80                     # e4m3 has NaN alone
    at = {w: ref.offsets(w, c.es, 16, D) for w in "kv"}
    for r in range(2):
        for pos in range(int(c.kv[r]), len(c.table[r]) * 16):
            page = c.table[r, pos // 16]
            if page < c.pages:
                for h in range(2):
                    c.kbits[page, h].reshape(-1)[at["k"][pos % 16]] = 0x7F if e4m3 else 0x7FC0
                    c.vbits[page, h].reshape(-1)[at["v"][pos % 16]] = inf
                    if e4m3:
                        c.ks[page, h, pos % 16], c.vs[page, h, pos % 16] = np.inf, np.nan
    first = int(c.q_start[1])
    c.mask[first:first + n] = [1 << i for i in range(n)]  # request 1: each node sees itself
    c.mask[first + 3] |= 1 << 1
    for node, d, what in ((1, 5, inf), (1, 9, 0x7F if e4m3 else 0x7FC0), (n - 1, 2, inf if e4m3 else inf - 0x8000)):
        page = c.table[1, node // 16]
        c.vbits[page, 1].reshape(-1)[at["v"][node % 16, d]] = what
    c.call().check()
    got = values(raw(c.out))[first:]
    assert np.isfinite(got[[0, 2]]).all() and not np.isfinite(got[1, G:, 5]).any() and not np.isfinite(got[3, G:, 9]).any()
    if e4m3:                                           # an infinite scale of a node that others do not see
        c.vbits[c.table[1, 0], 0].reshape(-1)[at["v"][2]] = 0x38
        c.vs[c.table[1, 0], 0, 2] = np.inf
        c.call().check()
        got = values(raw(c.out))[first:]
        assert np.isinf(got[2, :G]).all() and np.isfinite(got[[0, 1], :G]).all()


def test_attention_extreme_scores(tl):
    """Scores far apart (weights that underflow) and a scale of the caller's."""
    c = Case(tl, [(5, 300), (1, 700)], 1, 2, 128, False, 16, seed=13, qscale=60.0)
    c.call().check()
    c.scale = 0.37
    c.call().check()


def test_attention_strided_queries(tl, torch):
    """q as a column range of a wider tensor; out and lse of the requests alone are written."""
    c = Case(tl, [(3, 50), (2, 9)], 2, 3, 64, False, 16, seed=14)
    wide = torch.zeros((c.T, 6 * 64 + 128), dtype=torch.bfloat16, device=c.d)
    wide[:, 64:64 + 384] = bf16_dev(c.q.reshape(c.T, -1), c.d)
    c.call(q=wide[:, 64:64 + 384].unflatten(1, (6, 64))).check()
    c.q_start = np.array([0, 3, 3], dtype=np.int32)     # request 1 has no tokens now
    c.kv[1] = 9
    c.call()
    assert (values(raw(c.out))[3:] == 776.0).all() and (c.lse[3:] == 777.0).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_cache_beyond_32_bits(tl, torch, e4m3):
    """Pages whose elements lie past 2^32 bytes (and 2^31 elements) of the cache."""
    d, D, H, block = dev(), 128, 8, 64
    small = Case(tl, [(2, 190), (1, 60)], H, 2, D, e4m3, block, seed=15)
    page_bytes = H * block * D * small.es
    shift = (1 << 32) // page_bytes + 5
    pages = shift + small.pages
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k, v, ks, vs = tl.kv_cache(pages, H, block, D, dtype=kind, device=d)
    bits = torch.uint8 if e4m3 else torch.int16
    k.view(bits)[shift:] = to_dev(small.kbits, d)
    v.view(bits)[shift:] = to_dev(small.vbits, d)
    if e4m3:
        ks[shift:], vs[shift:] = to_dev(small.ks, d), to_dev(small.vs, d)
    small.call(k_cache=k, v_cache=v, k_scale=ks, v_scale=vs,
               block_table=to_dev(np.where(small.table < small.pages, small.table + shift, small.table), d)).check()
    # the same rows, written there
    rows = randn_bf16(np.random.default_rng(1), (4, H, D))
    slots = (pages - 1) * block + np.array([5, 6, 7, 40])
    tl.kv_write(bf16_dev(rows, d), bf16_dev(rows, d), to_dev(slots.astype(np.int64), d), k, v, k_scale=ks, v_scale=vs)
    page = values(raw(v[pages - 1:]))[0]
    got = np.stack([page[h].reshape(-1)[ref.offsets("v", small.es, block, D)] for h in range(H)], 1)[[5, 6, 7, 40]]
    if e4m3:
        got = got * vs[pages - 1].cpu().numpy().T[[5, 6, 7, 40]][..., None]
    assert (np.abs(got - rows) <= (2.0 ** -4 if e4m3 else 0) * np.abs(rows) + (2.0 ** -10 * 0.02 if e4m3 else 0)).all()


# --------------------------------------------------------------------------- tree_verify
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V,sizes", [(1, [1]), (7, [3, 1]), (1000, [64, 1, 0, 17]), (32003, [5] * 40), (248320, [9, 2]),
                                     (4099, [100, 3, 65, 1])])
def test_tree_verify(tl, torch, V, sizes, kind):
    announce(f"tree_verify V={V} sizes={sizes[:6]} {kind}")
    d, rng = dev(), np.random.default_rng(V)
    T = sum(sizes) + 2                                     # two rows that belong to no request
    x = ref.bf16(np.round(rng.standard_normal((T, V)) * 4) / 4)  # many ties
    x[rng.random(T) < 0.1] = -np.inf
    if V > 3:
        x[0, V // 2] = np.nan
        x[1, 1:3] = [0.0, -0.0]
    want = rng.integers(0, V, T)
    for t in range(2, T):
        if rng.random() < 0.7:
            x[t, want[t]] = 7.5
    parents = np.concatenate([np.where(rng.random(n) < 0.05, -1, np.where(rng.random(n) < 0.6, np.arange(n) - 1,
                              (rng.random(n) * np.arange(n)).astype(int))) for n in sizes] + [[0, 0]]).astype(np.int32)
    q_start = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    _, _, _, target = ref.verify(x, np.zeros(T, int), np.full(T, -1), [0, 0])
    draft = rng.integers(0, V, T).astype(np.int32)
    for r, n in enumerate(sizes):
        for i in range(1, n):
            p = parents[q_start[r] + i]
            if p >= 0 and rng.random() < 0.75:
                draft[q_start[r] + i] = target[q_start[r] + p]
    wide = torch.zeros((T, V + 5), dtype=torch.float32 if kind == "f32" else torch.bfloat16, device=d)
    wide[:, 3:V + 3] = torch.from_numpy(x).float().to(wide.dtype).to(d)
    for logits in (wide[:, 3:V + 3], wide[:, 3:V + 3].contiguous()):
        for width in (64, 2):
            got = tl.tree_verify(logits, to_dev(draft, d), to_dev(parents, d), to_dev(q_start, d), path_width=width)
            torch.cuda.synchronize()
            exp = ref.verify(x, draft, parents, q_start, width)
            for g, w, name in zip(got, exp, ("accepted", "path", "next", "target")):
                np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)


# --------------------------------------------------------------------------- kv_commit
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,H,block,layers", [(64, 1, 16, None), (128, 3, 32, 2), (256, 2, 16, 3)])
def test_kv_commit(tl, torch, D, H, block, layers, e4m3):
    announce(f"kv_commit D={D} H={H} block={block} layers={layers} e4m3={e4m3}")
    d, rng = dev(), np.random.default_rng(D)
    ctx = np.array([0, 5, 15, 33, 10, 3, 200, 7], dtype=np.int32)
    new = np.array([9, 64, 20, 1, 40, 6, 100, 30], dtype=np.int32)
    kv = ctx + new
    kv[5] = 0                                              # not served
    R = len(ctx)
    width = int(-(-(ctx + new).max() // block))
    pages = R * width + 2
    table = rng.permutation(pages)[:R * width].reshape(R, width).astype(np.int32)
    table[4, 1] = -1                                       # a bad page
    path = np.full((R, 64), -1, dtype=np.int32)
    accepted = np.zeros(R, dtype=np.int32)
    for r in range(R):
        k = min(int(new[r]), [4, 64, 12, 1, 20, 3, 100, 8][r])
        accepted[r] = k
        m = min(k, 64)
        path[r, :m] = np.concatenate([[0], 1 + np.sort(rng.permutation(min(int(new[r]), 64) - 1)[:m - 1])])
    path[7, :8] = [0, 29, 1, 40, 3, 2, 9, -5]              # entries that do not move a row forward inside the request
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    caches = tl.kv_cache(pages, H, block, D, dtype=kind, layers=layers, device=d)
    for c in caches[:2]:
        c.view(torch.uint8).copy_(torch.randint(0, 256, c.view(torch.uint8).shape, dtype=torch.uint8, device=d))
    for c in caches[2:]:
        if c is not None:
            c.copy_(torch.rand(c.shape, device=d))
    before = [None if c is None else (raw(c) if i < 2 else c.cpu().numpy()).copy() for i, c in enumerate(caches)]
    got = tl.kv_commit(to_dev(accepted, d), to_dev(path, d), to_dev(ctx, d), to_dev(kv, d), to_dev(table, d), *caches)
    torch.cuda.synchronize()
    moves, ctx_out = ref.commit_moves(accepted, path, ctx, kv, table, pages, block)
    np.testing.assert_array_equal(got.cpu().numpy(), ctx_out)
    es = 1 if e4m3 else 2
    at = [ref.offsets(w, es, block, D) for w in "kv"]
    for i, c in enumerate(caches):
        if c is None:
            continue
        want = before[i].copy().reshape((-1,) + before[i].shape[-4 if i < 2 else -3:])
        old = before[i].reshape(want.shape)
        for _, pa, ta, pb, tb in moves:
            if i < 2:
                w = want.reshape(want.shape[:3] + (-1,))
                o = old.reshape(w.shape)
                w[:, pb][..., at[i][tb]] = o[:, pa][..., at[i][ta]]
            else:
                want[:, pb, :, tb] = old[:, pa, :, ta]
        now = raw(c) if i < 2 else c.cpu().numpy()
        np.testing.assert_array_equal(now.reshape(want.shape), want)


# --------------------------------------------------------------------------- streams and graphs
def test_step_on_another_stream_and_in_a_graph(tl, torch):
    """A whole step (plan, write, attention, verification, commit) captured once and replayed with new
    lengths and tokens, on a stream of its own, against the same calls made eagerly."""
    d, rng = dev(), np.random.default_rng(21)
    R, T, H, G, D, block, V, width = 3, 40, 2, 4, 64, 16, 1003, 8
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=d)
    kc, vc, ks, vs = tl.kv_cache(R * width + 4, H, block, D, dtype=torch.float8_e4m3fn, device=d)
    state = dict(ctx=i32([0] * R), new=i32([0] * R), owned=i32([0] * R), table=i32(np.zeros((R, width))),
                 free=i32(rng.permutation(R * width + 4)), head=i32([0]), parents=i32([-1] * T), draft=i32([0] * T))
    qkv = torch.zeros((T, (G + 2) * H * D), dtype=torch.bfloat16, device=d)
    logits = torch.zeros((T, V), dtype=torch.bfloat16, device=d)
    cs = torch.rand((512, 32), device=d)
    out, lse = torch.empty((T, G * H, D), dtype=torch.bfloat16, device=d), torch.empty((T, G * H), device=d)

    def step():
        q_start, kv, slots, pos, mask, owned, head = tl.step_plan(
            state["ctx"], state["new"], state["owned"], state["table"], state["free"], state["head"], T, block,
            parents=state["parents"])
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([G * H * D, H * D, H * D], 1))
        q = tl.kv_write(k, v, slots, kc, vc, ks, vs, q=q, positions=pos, cos_sin=cs)
        tl.tree_attention(q, kc, vc, state["table"], q_start, kv, tree_mask=mask, k_scale=ks, v_scale=vs, max_nodes=20,
                          out=out, lse=lse)
        acc, path, nxt, target = tl.tree_verify(logits, state["draft"], state["parents"], q_start)
        ctx = tl.kv_commit(acc, path, state["ctx"], kv, state["table"], kc, vc, ks, vs)
        return q_start, kv, slots, pos, mask, owned, head, acc, path, nxt, target, ctx

    def inputs(seed):
        g = np.random.default_rng(seed)
        new = g.integers(1, 13, R)
        par = np.concatenate([(g.random(n) * np.arange(n)).astype(int) - (np.arange(n) == 0) for n in new] + [np.zeros(T, int)])[:T]
        state["ctx"].copy_(i32(g.integers(0, 90, R)))
        state["owned"].copy_(i32(-(-state["ctx"].cpu().numpy() // block)))
        state["new"].copy_(i32(new))
        state["parents"].copy_(i32(par))
        state["draft"].copy_(i32(g.integers(0, 4, T)))
        state["table"].copy_(i32(np.arange(R * width).reshape(R, width)))
        state["head"].copy_(i32([0]))
        state["free"].copy_(i32((np.arange(R * width + 4) * 7) % (R * width + 4)))
        qkv.copy_(torch.from_numpy(g.standard_normal(qkv.shape)).to(d).to(torch.bfloat16))
        logits.copy_(torch.from_numpy(g.integers(0, 3, logits.shape)).to(d).to(torch.bfloat16))
        for c in (kc, vc):
            c.view(torch.uint8).copy_(torch.from_numpy(g.integers(0, 0x60, c.shape, dtype=np.uint8)).to(d))
        for c in (ks, vs):
            c.fill_(0.01)
        out.zero_()
        lse.zero_()

    def result(r):
        return [x.clone() for x in r] + [out.clone(), lse.clone()] + [c.view(torch.uint8).clone() for c in (kc, vc)] + [ks.clone(), vs.clone()]

    announce("step eagerly, then captured and replayed")
    side = torch.cuda.Stream(d)
    eager = []
    for seed in range(4):
        inputs(seed)
        side.wait_stream(torch.cuda.current_stream(d))
        with torch.cuda.stream(side):
            r = step()
        torch.cuda.current_stream(d).wait_stream(side)
        eager.append(result(r))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        r = step()
    for seed in (0, 1, 2, 3, 1):
        inputs(seed)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        announce(f"  replay {seed}")
        for n, (a, b) in enumerate(zip(result(r), eager[seed])):
            assert torch.equal(a, b), f"output {n}"


FORMS = [(64, False, 4, "bf16_split16"), (64, False, 16, "bf16_split32"), (64, False, 17, "bf16_share128"),
         (128, False, 4, "bf16_split16"), (128, False, 8, "bf16_split32"), (128, False, 16, "bf16_share64"),
         (128, False, 17, "bf16_share128"), (256, False, 8, "bf16_split16"), (256, False, 9, "bf16_share128"),
         (64, True, 4, "e4m3_split16"), (64, True, 64, "e4m3_split32"), (64, True, 65, "e4m3_share128"),
         (128, True, 4, "e4m3_split16"), (128, True, 64, "e4m3_split32"), (128, True, 65, "e4m3_share128"),
         (256, True, 4, "e4m3_split16"), (256, True, 8, "e4m3_split16"), (256, True, 9, "e4m3_share128")]


@pytest.mark.parametrize("D,e4m3,nodes,form", FORMS)
def test_attention_each_form(tl, D, e4m3, nodes, form):
    """Both sides of each border between the kernel's forms (4 query heads a cache head), with trees that fill a
    block of rows and trees that do not, bad pages, empty rows and values that are not finite beside each tree."""
    reqs = [(min(nodes, 64), 150), (1, 700), (3, 0), (min(nodes, 64) // 2, 300), (nodes, 65)]
    c = Case(tl, reqs, 2, 4, D, e4m3, 32, seed=nodes + D)
    c.table[1, 4] = -1
    c.mask[c.q_start[2]:c.q_start[2] + 3] = [1, 0, 5]    # a node that sees nothing: there is no context either
    nan = 0x7F if e4m3 else 0x7FC0
    at = {w: ref.offsets(w, c.es, 32, D) for w in "kv"}
    for r in range(len(reqs)):                           # tokens past the end of each last page
        for pos in range(int(c.kv[r]), -(-int(c.kv[r]) // 32) * 32):
            c.kbits[c.table[r, pos // 32], :].reshape(2, -1)[:, at["k"][pos % 32]] = nan
            c.vbits[c.table[r, pos // 32], :].reshape(2, -1)[:, at["v"][pos % 32]] = nan
    c.vbits[c.table[2, 0], 1].reshape(-1)[at["v"][2, 7]] = nan   # seen by its own node alone
    c.call().check()
    assert tl.last_kernel_name() == "tree_attention_" + form
    got = values(raw(c.out))[c.q_start[2]:]
    assert np.isnan(got[2, 4:, 7]).all() and np.isfinite(got[:2]).all() and (got[1] == 0).all()


@pytest.mark.parametrize("D,hint", [(64, 1), (128, 40), (256, 12)])
def test_attention_requests_out_of_order(tl, D, hint):
    """Request starts that do not ascend: nothing is attended to, and nothing written."""
    c = Case(tl, [(3, 20), (4, 200), (5, 40)], 1, 4, D, False, 16, seed=21)
    c.q_start = np.array([0, 7, 3, 12], dtype=np.int32)
    c.call(max_nodes=hint)
    assert (values(raw(c.out)) == 776.0).all() and (c.lse == 777.0).all()
