"""Speculative-decoding operators without a GPU: the cache's element order, the
plain definitions on cases worked out by hand, and every refusal of the C ABI and
of the binding.  Every call below is rejected by the host checks (or is a zero-size
no-op) before any HIP call."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest

import oracle.speculative as ref
import quantized_gemv_gemm_amd as tl

pytestmark = pytest.mark.skipif(not os.path.exists(tl.LIB_PATH), reason="libtl.so not built")


def P(n):
    """A 4 GiB-spaced fake address, never dereferenced."""
    return ctypes.c_void_p((n + 1) << 32)


ODD = ctypes.c_void_p((77 << 32) + 2)


# --------------------------------------------------------------------------- layout
@pytest.mark.parametrize("code,bytes_", [(tl.TL_BF16, 2), (tl.TL_E4M3, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("which", ["k", "v"])
def test_offsets_match_the_description(which, D, code, bytes_):
    L, H, block = tl.lib(), 3, 32
    seen = set()
    for head in (0, 2):
        for token in range(block):
            for d in range(D):
                got = L.tl_kv_offset("kv".index(which), code, H, D, block, 5, head, token, d)
                assert got == ref.offset(which, bytes_, H, D, block, 5, head, token, d)
                seen.add(got)
    assert len(seen) == 2 * block * D  # no two elements share a place
    lo = 5 * H * block * D
    assert all(lo <= s < lo + H * block * D for s in seen)


def test_offset_passes_32_bits_and_refuses():
    L = tl.lib()
    assert L.tl_kv_offset(0, 0, 8, 128, 64, 1 << 20, 7, 63, 127) > 1 << 36
    bad = [(2, 0, 8, 128, 64, 0, 0, 0, 0), (0, 1, 8, 128, 64, 0, 0, 0, 0), (0, 0, 0, 128, 64, 0, 0, 0, 0),
           (0, 0, 8, 96, 64, 0, 0, 0, 0), (0, 0, 8, 128, 48, 0, 0, 0, 0), (0, 0, 8, 128, 64, -1, 0, 0, 0),
           (0, 0, 8, 128, 64, 0, 8, 0, 0), (0, 0, 8, 128, 64, 0, 0, 64, 0), (0, 0, 8, 128, 64, 0, 0, 0, 128)]
    for args in bad:
        assert L.tl_kv_offset(*args) == -1, args
    torch = pytest.importorskip("torch")
    assert tl.kv_offset("v", torch.bfloat16, 1, 64, 16, 0, 0, 9, 17) == ref.offset("v", 2, 1, 64, 16, 0, 0, 9, 17)
    with pytest.raises(ValueError):
        tl.kv_offset("x", torch.bfloat16, 1, 64, 16, 0, 0, 0, 0)


# --------------------------------------------------------------------------- the plain definitions, by hand
def test_e4m3_numbers():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = ref.e4m3_value(codes)
    assert np.array_equal(got, want, equal_nan=True)
    x = np.concatenate([got[np.isfinite(got)], np.random.default_rng(0).uniform(-450, 450, 5000),
                        (got[:126] + got[1:127]) / 2, np.random.default_rng(1).uniform(-0.03, 0.03, 3000)])
    t = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_code(x.astype(np.float32)), t)


def test_plan_by_hand():
    # pages of 16; three free pages; request 1 needs two, request 2 one more than is left
    table = np.array([[4, 0, 0], [0, 0, 0], [6, 0, 0], [0, 0, 0]])
    free = np.array([9, 8, 7])
    got = ref.step_plan(np.array([14, 0, 16, 3]), np.array([3, 20, 1, 46]), np.array([1, 0, 1, 0]), table, free, 0, 75, 16,
                        np.array([-1, 0, 0] + [-1] + list(range(19)) + [-1] + [-1] * 46 + [0] * 5))
    q_start, kv, slots, pos, mask, owned, head, out = got
    assert q_start.tolist() == [0, 3, 23, 24, 70]
    assert kv.tolist() == [17, 20, 0, 0] and owned.tolist() == [2, 2, 1, 0] and head == 3
    assert out.tolist() == [[4, 9, 0], [8, 7, 0], [6, 0, 0], [0, 0, 0]]
    assert slots[:5].tolist() == [4 * 16 + 14, 4 * 16 + 15, 9 * 16, 8 * 16, 8 * 16 + 1]
    assert pos[:4].tolist() == [14, 15, 15, 0] and mask[:3].tolist() == [1, 3, 5]
    assert mask[22] == (1 << 20) - 1 and (slots[23:] == -1).all() and (pos[70:] == 0).all()


def test_verify_by_hand():
    logits = np.zeros((6, 10))
    for t, v in enumerate([3, 7, 1, 2, 9, 4]):
        logits[t, v] = 1.0
    #        0
    #     1(5)  2(3)        target(0) = 3: node 2, target(2) = 1: the first of nodes 3 and 4
    #          3(1) 4(1)
    draft, parents = [0, 5, 3, 1, 1, 2], [-1, 0, 0, 2, 2, 4]
    acc, path, nxt, target = ref.verify(logits, draft, parents, [0, 6])
    assert target.tolist() == [3, 7, 1, 2, 9, 4]
    assert acc.tolist() == [3] and path[0, :4].tolist() == [0, 2, 3, -1] and nxt.tolist() == [2]
    x = np.array([[1.0, np.nan, 5.0], [0.0, -0.0, 0.0], [-np.inf] * 3, [2.0, 5.0, 5.0]])
    assert ref.verify(x, [0] * 4, [-1] * 4, [0, 4])[3].tolist() == [1, 0, 0, 1]


def test_commit_and_attention_by_hand():
    moves, ctx = ref.commit_moves([3, 2], np.array([[0, 2, 3], [0, 1, -1]]), [15, 4], [19, 6],
                                  np.array([[1, 0], [2, -1]]), 3, 16)
    assert moves == [(0, 0, 1, 0, 0), (0, 0, 2, 0, 1)] and ctx.tolist() == [18, 6]
    q, k, v = np.ones((2, 1, 1)), np.zeros((3, 1)), np.array([[1.0], [3.0], [8.0]])
    out, lse = ref.attention(q, k, v, np.ones(3, bool), 2, [1, 3], 1.0)
    assert out[:, 0, 0].tolist() == [2.0, 4.0] and np.allclose(lse[:, 0], np.log([2, 3]))
    out, lse = ref.attention(q, k, v, np.array([False, True, True]), 2, [0, 1], 1.0)
    assert out[:, 0, 0].tolist() == [0.0, 3.0] and lse[0, 0] == -np.inf


# --------------------------------------------------------------------------- refusals
def test_plan_rejections():
    L = tl.lib()

    def call(ctx=P(0), new=P(1), owned=P(2), R=4, table=P(3), width=8, block=16, free=P(4), nfree=9, head=P(5),
             parents=P(6), T=20, qs=P(7), kv=P(8), slots=P(9), pos=P(10), mask=P(11), oo=P(12), ho=P(13)):
        return L.tl_step_plan(ctx, new, owned, R, table, width, block, free, nfree, head, parents, T, qs, kv, slots,
                              pos, mask, oo, ho, None)
    for bad in (dict(R=-1), dict(R=4097), dict(T=-1), dict(T=1 << 31), dict(nfree=-1), dict(block=24), dict(block=8),
                dict(block=8192), dict(width=-1), dict(width=1 << 27)):
        assert call(**bad) == 2, bad
    for name in ("ctx", "new", "owned", "table", "free", "head", "qs", "kv", "slots", "pos", "mask", "oo", "ho"):
        assert call(**{name: None}) == 1, name
    for name in ("ctx", "new", "owned", "table", "free", "head", "parents", "qs", "kv", "slots", "pos", "mask", "oo", "ho"):
        assert call(**{name: ODD}) == 3, name
    assert call(slots=ctypes.c_void_p((78 << 32) + 4)) == 3
    for a, b in (("qs", P(0)), ("kv", P(1)), ("oo", P(2)), ("ho", P(5)), ("table", P(4)), ("slots", P(6)), ("pos", P(9)),
                 ("mask", P(10))):
        assert call(**{a: b}) == 8, a


def test_write_rejections():
    L = tl.lib()

    def call(k=P(0), ldk=512, v=P(1), ldv=512, slots=P(2), T=4, H=4, D=128, q=P(3), ldq=1024, Hq=8, pos=P(4), cs=P(5),
             most=100, rot=64, qo=P(6), kc=P(7), vc=P(8), ks=P(9), vs=P(10), dt=tl.TL_E4M3, pages=3, block=16):
        return L.tl_kv_write(k, ldk, v, ldv, slots, T, H, D, q, ldq, Hq, pos, cs, most, rot, qo, kc, vc, ks, vs, dt,
                             pages, block, None)
    for bad in (dict(T=-1), dict(D=96), dict(H=0), dict(block=20), dict(pages=0), dict(ldk=504), dict(ldv=511),
                dict(ldq=1000), dict(Hq=0), dict(rot=8), dict(rot=144), dict(most=0), dict(pages=1 << 30, H=65536, ldk=1 << 23, ldv=1 << 23)):
        assert call(**bad) == 2, bad
    assert call(dt=tl.TL_F32) == 4
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs", "qo", "pos"):
        assert call(**{name: None}) == 1, name
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs", "qo", "pos", "q", "cs"):
        assert call(**{name: ODD}) == 3, name
    assert call(ldk=516) == 3 and call(ldq=1028) == 3
    for name, at in (("kc", P(0)), ("vc", P(7)), ("qo", P(3)), ("ks", P(4)), ("vs", P(9))):
        assert call(**{name: at}) == 8, name
    assert call(T=0) == 0


def test_attention_rejections():
    L = tl.lib()
    need = L.tl_tree_attention_workspace_size(16, 4, 128, tl.TL_BF16)
    assert need > 0
    for bad in ((0, 4, 128, 0), (16, 0, 128, 0), (16, 65, 128, 0), (16, 4, 100, 0), (16, 4, 128, 1)):
        assert L.tl_tree_attention_workspace_size(*bad) == 0

    def call(q=P(0), ldq=1024, T=30, H=2, G=4, D=128, kc=P(1), vc=P(2), ks=P(3), vs=P(4), dt=tl.TL_E4M3, pages=9, block=16,
             table=P(5), width=4, R=2, qs=P(6), kv=P(7), mask=P(8), scale=0.1, nodes=16, out=P(9), lse=P(10), ws=P(11),
             wb=1 << 31):
        return L.tl_tree_attention(q, ldq, T, H, G, D, kc, vc, ks, vs, dt, pages, block, table, width, R, qs, kv, mask,
                                   scale, nodes, out, lse, ws, wb, None)
    for bad in (dict(T=-1), dict(R=-1), dict(R=5000), dict(G=0), dict(G=65), dict(D=32), dict(H=0), dict(block=17),
                dict(pages=0), dict(ldq=1016), dict(width=-1), dict(nodes=0), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(T=1 << 24, width=1 << 20)):
        assert call(**bad) == 2, bad
    assert call(dt=tl.TL_F32) == 4
    for name in ("q", "kc", "vc", "ks", "vs", "table", "qs", "kv", "out"):
        assert call(**{name: None}) == 1, name
    assert call(ws=None) == 7
    assert call(dt=tl.TL_BF16, wb=need - 1) == 7
    for name in ("q", "kc", "vc", "ks", "vs", "table", "qs", "kv", "out", "mask", "lse", "ws"):
        assert call(**{name: ODD}) == 3, name
    assert call(ldq=1028) == 3
    for name, at in (("out", P(0)), ("lse", P(7)), ("ws", P(1))):
        assert call(**{name: at}) == 8, name
    assert call(T=0) == 0 and call(R=0) == 0


def test_verify_rejections():
    L = tl.lib()
    assert L.tl_tree_verify_workspace_size(-1, 5) == 0 and L.tl_tree_verify_workspace_size(3, 0) == 0
    need = L.tl_tree_verify_workspace_size(17, 50000)
    assert need >= 17 * 8

    def call(x=P(0), dt=1, ld=50000, T=17, V=50000, draft=P(1), par=P(2), qs=P(3), R=2, acc=P(4), path=P(5), width=64,
             nxt=P(6), tgt=P(7), ws=P(8), wb=need):
        return L.tl_tree_verify(x, dt, ld, T, V, draft, par, qs, R, acc, path, width, nxt, tgt, ws, wb, None)
    assert call(dt=2) == 4
    for bad in (dict(T=-1), dict(V=0), dict(ld=49999), dict(R=-1), dict(R=4097), dict(width=0), dict(width=65)):
        assert call(**bad) == 2, bad
    for name in ("x", "draft", "par", "qs", "acc", "path", "nxt", "tgt"):
        assert call(**{name: None}) == 1, name
    assert call(ws=None) == 7 and call(wb=need - 1) == 7
    for name in ("x", "draft", "par", "qs", "acc", "path", "nxt", "tgt", "ws"):
        assert call(**{name: ODD}) == 3, name
    for name, at in (("tgt", P(0)), ("path", P(4)), ("ws", P(3))):
        assert call(**{name: at}) == 8, name
    assert call(T=0, R=0, wb=0) == 0


def test_commit_rejections():
    L = tl.lib()

    def call(acc=P(0), path=P(1), pw=64, ctx=P(2), kv=P(3), table=P(4), width=4, R=2, kc=P(5), vc=P(6), ks=P(7), vs=P(8),
             dt=tl.TL_E4M3, layers=2, pages=3, H=2, block=16, D=64, out=P(9)):
        return L.tl_kv_commit(acc, path, pw, ctx, kv, table, width, R, kc, vc, ks, vs, dt, layers, pages, H, block, D, out,
                              None)
    for bad in (dict(pw=0), dict(pw=65), dict(R=-1), dict(layers=0), dict(H=0), dict(block=15), dict(D=65), dict(pages=0),
                dict(width=-1), dict(R=4096, layers=4096, H=1024)):
        assert call(**bad) == 2, bad
    assert call(dt=1) == 4
    for name in ("acc", "path", "ctx", "kv", "table", "kc", "vc", "ks", "vs", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("acc", "path", "ctx", "kv", "table", "kc", "vc", "ks", "vs", "out"):
        assert call(**{name: ODD}) == 3, name
    for name, at in (("out", P(2)), ("kc", P(0)), ("vc", P(5)), ("ks", P(7 + 1))):
        assert call(**{name: at}) == 8, name
    assert call(R=0) == 0


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    k, v, _, _ = tl.kv_cache(2, 2, 16, 64, device="cpu")
    assert k.shape == (2, 2, 16, 64) and k.dtype is torch.bfloat16 and v.shape == k.shape
    e = tl.kv_cache(2, 2, 16, 64, dtype=torch.float8_e4m3fn, layers=3, device="cpu")
    assert e[0].shape == (3, 2, 2, 16, 64) and e[2].shape == (3, 2, 2, 16)
    with pytest.raises(TypeError):
        tl.kv_cache(2, 2, 16, 64, dtype=torch.float16, device="cpu")
    with pytest.raises(ValueError):
        tl.step_plan(i32(1), i32(1), i32(1), i32(1, 2), i32(3), i32(1), 4, 16)
    with pytest.raises(ValueError):
        tl.kv_write(x, x, torch.zeros(2, dtype=torch.int64), k, v)
    with pytest.raises(ValueError):
        tl.tree_attention(x, k, v, i32(1, 2), i32(2), i32(1))
    with pytest.raises(ValueError):
        tl.tree_verify(torch.zeros((2, 9)), i32(2), i32(2), i32(2))
    with pytest.raises(ValueError):
        tl.kv_commit(i32(1), i32(1, 4), i32(1), i32(1), i32(1, 2), k, v)
    with pytest.raises(TypeError):
        tl.tree_attention([1], k, v, i32(1, 2), i32(2), i32(1))
