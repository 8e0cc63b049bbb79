"""The token mixers of a hybrid decoder without a GPU: their plain definitions against each other and by hand, and every
refusal of the C ABI and of the binding (by the host checks, before any HIP call)."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest

import oracle.mixers as ref
import quantized_gemv_gemm_amd as tl

pytestmark = pytest.mark.skipif(not os.path.exists(tl.LIB_PATH), reason="libtl.so not built")


def P(n):
    """A 16 GiB-spaced fake address, never dereferenced."""
    return ctypes.c_void_p((n + 1) << 34)


ODD = ctypes.c_void_p((77 << 34) + 2)


# --------------------------------------------------------------------------- the definitions
def test_norm_and_turn_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    assert np.allclose(ref.normed(x, None, 0.0), x / 2.5) and np.allclose(ref.normed(x, np.arange(4.0), 0.0), [[[0, 1.6, 0, 0]]])
    cs = np.array([[1, 1, 0, 0], [0, 1, 1, 0], [1, -1, 0, 0]], dtype=np.float32)   # cos, cos, sin, sin at positions 0..2
    y = ref.turned(x, cs, np.array([[1], [2]]), [0, 1])
    assert y.tolist() == [[[0.0, -4.0, 3.0, 0.0]]]                                 # (3, 0) by 90, (4, 0) by 180 degrees
    assert ref.turned(x, cs, np.array([[9], [-1]]), [-5, 7]).tolist() == [[[3.0, 4.0, 0.0, 0.0]]]   # all clamped


def test_conv_by_hand():
    x, w = np.array([[1.0], [2.0], [4.0]]), np.array([[1.0, 10.0, 100.0]])
    silu = lambda v: v / (1 + np.exp(-v))
    out, after, _ = ref.short_conv(x, w, None, [0, 3], [5], [1], np.array([[[0.0], [0.0]], [[7.0], [8.0]]]), None, 0, 1, 0.0, np.zeros((3, 1)))
    assert np.allclose(out[:, 0], silu(np.array([187.0, 218.0, 421.0]))) and after[1, :, 0].tolist() == [2.0, 4.0]
    # a tree: 2's parent is 0
    out, after, _ = ref.short_conv(x, w, None, [0, 3], [5], [1], np.array([[[0.0], [0.0]], [[7.0], [8.0]]]), [1, 3, 5], 0, 1, 0.0, np.zeros((3, 1)))
    assert np.allclose(out[:, 0], silu(np.array([187.0, 218.0, 418.0]))) and after[1, :, 0].tolist() == [7.0, 8.0]


def test_delta_by_hand_and_as_a_tree():
    one = lambda *v: np.array(v, dtype=np.float64).reshape(-1, 1, 1)
    # S = 2; decay 1/2, step 1: S -> 1 + 1 (3 - 1) = 3, out = 3; then step 0: S = 1.5, out = 1.5 * 2
    out, after, _ = ref.delta_rule(one(1, 2), one(1, 1), one(3, 9), np.log([[0.5], [0.5]]), np.array([[1.0], [0.0]]), [0, 2], [9], [0],
                                   np.full((1, 1, 1, 1), 2.0), None, 1.0, np.zeros((2, 1, 1)))
    assert np.allclose(out[:, 0, 0], [3, 3]) and np.allclose(after, 1.5)
    rng = np.random.default_rng(0)
    T, Hk, Hv, Dk, Dv = 40, 2, 4, 8, 6
    q, k, v = (rng.standard_normal((T, h, n)) / 3 for h, n in ((Hk, Dk), (Hk, Dk), (Hv, Dv)))
    g, b = -rng.random((T, Hv)), rng.random((T, Hv))
    state = rng.standard_normal((2, Hv, Dk, Dv))
    args = ([0, 30, 40], [50, 10], [1, 0], state)
    chain = np.array([(1 << i + 1) - 1 for n in (30, 10) for i in range(n)], dtype=np.uint64)
    a, sa, _ = ref.delta_rule(q, k, v, g, b, *args, None, 1.0, np.zeros((T, Hv, Dv)))
    t, st, _ = ref.delta_rule(q, k, v, g, b, *args, chain, 1.0, np.zeros((T, Hv, Dv)))
    assert np.allclose(a, t) and np.array_equal(st, state) and not np.allclose(sa, state)
    done, _ = ref.delta_commit([30, 10], np.tile(np.arange(30), (2, 1)), *args[:3], k, v, g, b, state, np.zeros((T, 8)), np.zeros((2, 3, 8)))
    assert np.allclose(done, sa)
    # a branch's token gives what the chain of its ancestors gives
    words, line = np.array([1, 3, 5, 13, 19], dtype=np.uint64), [0, 2, 3]
    t, _, _ = ref.delta_rule(q[:5], k[:5], v[:5], g[:5], b[:5], [0, 5], [9], [1], state, words, 1.0, np.zeros((5, Hv, Dv)))
    a, _, _ = ref.delta_rule(q[line], k[line], v[line], g[line], b[line], [0, 3], [9], [1], state, None, 1.0, np.zeros((3, Hv, Dv)))
    assert np.allclose(t[3], a[2])


# --------------------------------------------------------------------------- refusals
def test_write_norm_rejections():
    L = tl.lib()

    def call(k=P(0), ldk=512, v=P(1), ldv=512, slots=P(2), T=4, H=4, D=128, q=P(3), ldq=2048, hq=256, Hq=8, qw=P(11), kw=P(12),
             eps=1e-6, pos=P(4), axes=3, axis=P(13), cs=P(5), most=100, rot=64, qo=P(6), kc=P(7), vc=P(8), ks=P(9), vs=P(10),
             dt=tl.TL_E4M3, pages=3, block=16):
        return L.tl_kv_write_norm(k, ldk, v, ldv, slots, T, H, D, q, ldq, hq, Hq, qw, kw, eps, pos, axes, axis, cs, most, rot, qo,
                                  kc, vc, ks, vs, dt, pages, block, None)
    for bad in (dict(T=-1), dict(D=96), dict(H=0), dict(block=20), dict(pages=0), dict(ldk=504), dict(ldv=511), dict(ldq=1912),
                dict(hq=120), dict(hq=1 << 31), dict(Hq=0), dict(rot=8), dict(rot=144), dict(most=0), dict(axes=0), dict(axes=17),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**bad) == 2, bad
    assert call(dt=tl.TL_F32) == 4
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs", "qo", "pos", "axis"):
        assert call(**{name: None}) == 1, name
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs", "qo", "pos", "q", "cs", "qw", "kw", "axis"):
        assert call(**{name: ODD}) == 3, name
    assert call(ldk=516) == 3 and call(ldq=2052) == 3 and call(hq=252, ldq=2048) == 3
    for name, at in (("kc", P(0)), ("vc", P(7)), ("qo", P(3)), ("ks", P(4)), ("vs", P(9)), ("kc", P(12)), ("qo", P(11)), ("ks", P(13))):
        assert call(**{name: at}) == 8, name
    assert call(T=0) == 0


def test_conv_rejections():
    L = tl.lib()

    def call(x=P(0), ldx=512, T=9, C=512, w=P(1), taps=4, bias=P(2), qs=P(3), kv=P(4), slots=P(5), R=2, mask=P(6), heads=2, dim=128,
             eps=1e-6, state=P(7), states=5, out=P(8), ldo=512):
        return L.tl_short_conv(x, ldx, T, C, w, taps, bias, qs, kv, slots, R, mask, heads, dim, eps, state, states, out, ldo, None)
    for bad in (dict(T=-1), dict(T=1 << 31), dict(C=0), dict(C=516), dict(C=(1 << 20) + 8, ldx=1 << 21, ldo=1 << 21), dict(ldx=504),
                dict(ldo=504), dict(taps=1), dict(taps=5), dict(R=-1), dict(R=4097), dict(heads=-1), dict(heads=5), dict(dim=32),
                dict(eps=-1.0), dict(eps=float("nan")), dict(states=-1), dict(states=1 << 31)):
        assert call(**bad) == 2, bad
    for name in ("x", "w", "qs", "kv", "slots", "state", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("x", "w", "bias", "qs", "kv", "slots", "mask", "state", "out"):
        assert call(**{name: ODD}) == 3, name
    assert call(ldx=516) == 3 and call(ldo=516) == 3
    for name, at in (("out", P(0)), ("state", P(1)), ("out", P(7)), ("state", P(4))):
        assert call(**{name: at}) == 8, name
    assert call(T=0) == 0 and call(R=0) == 0


def test_delta_rejections():
    L = tl.lib()
    size = L.tl_delta_rule_workspace_size
    assert size(64, 64, 16, 3, 128, 1, 0) == 0 and size(64, 64, 16, 3, 128, 64, 1) == 0      # one launch each
    assert size(100, 2, 16, 3, 128, 64, 0) == 0
    assert size(64, 64, 16, 3, 128, 65, 1) > 0 and size(100, 2, 16, 3, 128, 65, 0) > 0
    for bad in ((-1, 2, 1, 1, 64, 50, 0), (9, -1, 1, 1, 64, 50, 0), (9, 4097, 1, 1, 64, 50, 0), (9, 2, 0, 1, 64, 50, 0),
                (9, 2, 1, 1, 32, 50, 0), (9, 2, 1, 1, 64, 0, 0), (9, 2, 65536, 1, 64, 50, 0)):
        assert size(*bad) == 0, bad
    need = size(90, 2, 2, 3, 64, 80, 1)

    def call(q=P(0), ldq=128, k=P(1), ldk=128, v=P(2), ldv=192, a=P(3), lda=6, b=P(4), ldb=6, log=P(5), bias=P(6), T=90, Hk=2, G=3,
             Dk=64, Dv=32, qs=P(7), kv=P(8), slots=P(9), R=2, mask=P(10), scale=0.1, state=P(11), states=5, nodes=80, out=P(12),
             ws=P(13), wb=need):
        return L.tl_delta_rule(q, ldq, k, ldk, v, ldv, a, lda, b, ldb, log, bias, T, Hk, G, Dk, Dv, qs, kv, slots, R, mask, scale,
                               state, states, nodes, out, ws, wb, None)
    for bad in (dict(T=-1), dict(T=1 << 31), dict(R=-1), dict(R=4097), dict(Hk=0), dict(G=0), dict(Hk=300, G=300), dict(Dk=96),
                dict(Dk=256, ldq=1 << 10, ldk=1 << 10), dict(Dv=8), dict(Dv=40), dict(Dv=65552, ldv=1 << 20), dict(ldq=120), dict(ldk=120),
                dict(ldv=184), dict(lda=5), dict(ldb=5), dict(ldv=1 << 31), dict(states=-1), dict(nodes=0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(states=1 << 30, G=100, Dv=4096, ldv=1 << 20, lda=300, ldb=300),
                dict(R=4096, Hk=60, G=1000, Dv=160, ldq=1 << 14, ldk=1 << 14, ldv=1 << 24, lda=1 << 17, ldb=1 << 17, states=1)):
        assert call(**bad) == 2, bad
    for name in ("q", "k", "v", "a", "b", "qs", "kv", "slots", "state", "out", "log", "bias"):
        assert call(**{name: None}) == 1, name
    assert call(ws=None) == 7 and call(wb=need - 1) == 7
    for name in ("q", "k", "v", "a", "b", "qs", "kv", "slots", "state", "out", "log", "bias", "mask", "ws"):
        assert call(**{name: ODD}) == 3, name
    assert call(ldq=132) == 3 and call(ldk=132) == 3 and call(ldv=196) == 3
    for name, at in (("out", P(0)), ("state", P(2)), ("ws", P(11)), ("out", P(5)), ("state", P(8))):
        assert call(**{name: at}) == 8, name
    assert call(T=0) == 0 and call(R=0) == 0


def test_commit_rejections():
    L = tl.lib()

    def call(acc=P(0), path=P(1), width=9, qs=P(2), kv=P(3), slots=P(4), R=2, T=40, layers=3, k=P(5), ldk=128, k_layer=128 * 40, v=P(6),
             ldv=192, v_layer=192 * 40, a=P(7), lda=6, a_layer=240, b=P(8), ldb=6, b_layer=240, log=P(9), bias=P(10), Hk=2, G=3, Dk=64,
             Dv=32, state=P(11), states=5, x=P(12), ldx=448, x_layer=448 * 40, C=448, taps=4, conv=P(13)):
        return L.tl_delta_commit(acc, path, width, qs, kv, slots, R, T, layers, k, ldk, k_layer, v, ldv, v_layer, a, lda, a_layer, b, ldb,
                                 b_layer, log, bias, Hk, G, Dk, Dv, state, states, x, ldx, x_layer, C, taps, conv, None)
    for bad in (dict(T=-1), dict(R=-1), dict(R=4097), dict(layers=0), dict(layers=4097), dict(width=0), dict(width=65), dict(Hk=0),
                dict(Dk=32), dict(Dv=24), dict(ldk=120), dict(ldv=184), dict(lda=5), dict(ldb=5), dict(k_layer=-1), dict(v_layer=-8),
                dict(a_layer=-1), dict(b_layer=-1), dict(x_layer=-8), dict(k_layer=1 << 46), dict(C=4), dict(ldx=440), dict(taps=5),
                dict(states=-1), dict(states=1 << 30, layers=4096, G=100, Dv=320, ldv=1 << 20, lda=200, ldb=200),
                dict(R=4096, layers=4096, G=100, lda=200, ldb=200, ldv=8192)):
        assert call(**bad) == 2, bad
    for name in ("acc", "path", "qs", "kv", "slots", "k", "v", "a", "b", "log", "bias", "state", "conv"):
        assert call(**{name: None}) == 1, name
    for name in ("acc", "path", "qs", "kv", "slots", "k", "v", "a", "b", "log", "bias", "state", "x", "conv"):
        assert call(**{name: ODD}) == 3, name
    assert call(k_layer=5124) == 3 and call(ldx=452) == 3
    for name, at in (("state", P(5)), ("conv", P(12)), ("conv", P(11)), ("state", P(1))):
        assert call(**{name: at}) == 8, name
    assert call(T=0) == 0 and call(R=0) == 0


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    k, v, _, _ = tl.kv_cache(2, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        tl.kv_write_norm(x, x, torch.zeros(2, dtype=torch.int64), k, v)
    with pytest.raises(ValueError):
        tl.short_conv(x[:, 0], torch.zeros(64, 4), i32(2), i32(1), i32(1), torch.zeros((1, 3, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        tl.delta_rule(x, x, x, torch.zeros(2, 2), torch.zeros(2, 2), i32(2), i32(1), i32(1), torch.zeros(1, 2, 64, 64))
    with pytest.raises(ValueError):
        tl.delta_commit(i32(1), i32(1, 4), i32(2), i32(1), i32(1), x, x, torch.zeros(2, 2), torch.zeros(2, 2), torch.zeros(1, 2, 64, 64))
    with pytest.raises(TypeError):
        tl.short_conv([1], torch.zeros(64, 4), i32(2), i32(1), i32(1), None)


def test_the_plain_hybrid_decoder_goes_on_where_it_stopped():
    """Its states and rows carry everything: a history in parts is the history; a token lost from the states shows in
    every later logit and in none before."""
    from oracle.hybrid import Decoder
    rng = np.random.default_rng(0)
    Hk, Hv, Dk, Dv, taps = 2, 4, 32, 256, 3
    C = 2 * Hk * Dk + Hv * Dv
    linear = lambda K, N: (rng.integers(-1, 2, (N, K)).astype(np.int8), np.full((N, K // 128), (1.5 / K) ** 0.5, np.float16))
    layer = lambda N, K: [linear(1024, N), linear(K, 1024), linear(1024, 2048), linear(1024, 1024)]
    angle = rng.uniform(0, 6, (64, 16))
    w = dict(embed=rng.standard_normal((32, 1024)), taps=rng.standard_normal((2, C, taps)), gates=rng.standard_normal((2, 1024, 2 * Hv)) / 32,
             a_log=rng.standard_normal((2, Hv)) - 2, dt_bias=rng.standard_normal((2, Hv)), q_weight=rng.standard_normal((1, 128)),
             k_weight=rng.standard_normal((1, 128)), cos_sin=np.concatenate([np.cos(angle), np.sin(angle)], 1))
    d = Decoder(w, [layer(C, Hv * Dv) for _ in range(2)], [layer(10 * 128, 1024)], linear(1024, 32), (8, 1, 128, Hk, Hv, Dk, Dv), True)
    tokens = rng.integers(0, 32, 20).tolist()
    y, _ = d.rows(tokens, None)
    a, state = d.rows(tokens[:7], None)
    b, _ = d.rows(tokens[7:], state)
    np.testing.assert_allclose(np.concatenate([a, b]), y, atol=1e-9)
    assert d.greedy(tokens, 2)[0] == np.argmax(y[-1])
    far = np.sqrt(((d.rows(tokens, None, {9})[0] - y) ** 2).mean(-1))
    assert (far[:10] == 0).all() and (far[10:] > 0.1).all()
