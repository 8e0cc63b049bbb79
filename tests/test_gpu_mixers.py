"""The token mixers of a hybrid decoder (normed cache write, short convolution, gated delta rule, commit of its states)
on the GPU against their plain definitions in 64 bits (oracle/mixers.py).  Moved rows are exact; computed values stay
within bounds counted from the roundings the kernels make."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.mixers as ref
import oracle.speculative as spec
from gpu_common import announce, dev, to_dev

pytestmark = pytest.mark.gpu

BF16_HALF = 2.0 ** -8      # half a step of bfloat16, relative
F32_HALF = 2.0 ** -24
# States, in the 2-norm: every value is a chain of sums of up to 128 terms (S^T k) and 64 (a chunk's u), of f32 roundings
# with independent signs: 14 half steps for each sum and the few roundings around it, over the chunks that the state
# remembers.  With decays and steps of these tests that is at most 16 of them, 4 in the root: 56.
STATE_TOL = 64 * F32_HALF
# of each form of the delta rule a max_nodes that takes it
FORMS = {"step": 1, "one chunk": 64, "chunks": 1000, "trees": 64, "trees and chunks": 130}
KERNEL = {"step": "delta_step", "one chunk": "delta_chunk", "trees": "delta_tree"}
# P and S^T q reach the output as two parts of 8 bits each, the first cut off: 2^-16 of each term, in both operands
PARTS = 2.0 ** -14


@pytest.fixture(scope="module")
def tl():
    import quantized_gemv_gemm_amd as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def torch():
    import torch
    return torch


def f64(t):
    return t.double().cpu().numpy()


def bits(t):
    import torch
    kind = {2: torch.int16, 4: torch.int32, 1: torch.uint8}[t.element_size()]
    return t.contiguous().view(kind).cpu().numpy()


def bf16_dev(x, d):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(torch.bfloat16).to(d)


def f32_dev(x, d):
    return to_dev(np.asarray(x, dtype=np.float32), d)


# --------------------------------------------------------------------------- kv_write_norm
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,H,Hq,D,rot,axes,gated,weights,block,first", [
    (1, 1, 1, 64, 0, 1, False, False, 16, 0), (1, 4, 24, 256, 64, 1, True, True, 16, 5), (7, 2, 6, 128, 128, 3, False, True, 16, 3),
    (16, 1, 8, 128, 64, 2, True, True, 32, 0), (33, 3, 3, 64, 32, 3, True, False, 64, 15), (100, 2, 5, 256, 256, 4, False, True, 64, 9),
    (50, 8, 0, 128, 16, 1, False, True, 128, 120), (257, 1, 2, 64, 64, 3, False, True, 32, 30)])
def test_kv_write_norm(tl, torch, T, H, Hq, D, rot, axes, gated, weights, block, first, e4m3):
    announce(f"kv_write_norm T={T} H={H} Hq={Hq} D={D} rot={rot} axes={axes} gated={gated} block={block} e4m3={e4m3}")
    d, rng = dev(), np.random.default_rng(T * 7 + D + rot + axes)
    wide = 2 * D if gated else D
    x = spec.bf16(rng.standard_normal((T, Hq * wide + 2 * H * D + 8)) * np.exp(2 * rng.standard_normal((T, 1))))
    x[rng.random(T) < 0.1] = 0.0                                       # rows of zeros: eps alone is their length
    xd = bf16_dev(x, d)
    q, qd = (x[:, :Hq * wide].reshape(T, Hq, wide)[..., :D], xd[:, :Hq * wide].unflatten(1, (Hq, wide))[..., :D]) if Hq else (None, None)
    part = lambda i: (x[:, Hq * wide + i * H * D:][:, :H * D].reshape(T, H, D),
                      xd[:, Hq * wide + i * H * D:][:, :H * D].unflatten(1, (H, D)))
    (k, kd), (v, vd) = part(0), part(1)
    wq, wk = (rng.standard_normal(D).astype(np.float32) for _ in "qk") if weights else (None, None)
    pages = -(-(T + first) // block) + 2
    order, at = rng.permutation(pages), np.arange(T) + first
    slots = order[at // block] * block + at % block
    skip = rng.random(T) < 0.1
    slots = np.where(skip, rng.choice([-1, -5, pages * block, 1 << 40], T), slots).astype(np.int64)
    positions = rng.integers(-2, 5000, (axes, T)).astype(np.int32)
    axis_of = rng.integers(-1, axes + 1, rot // 2).astype(np.int32) if axes > 1 else None   # clamped to the axes
    cs = None
    if rot:
        a = rng.uniform(0, 6.28, (4096, rot // 2))
        cs = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    eps = 1e-5
    kc, vc, ks, vs = tl.kv_cache(pages, H, block, D, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device=d)
    for c in (kc, vc):
        c.view(torch.uint8).fill_(0x5A)
    if e4m3:
        ks.fill_(-3.0)
        vs.fill_(-3.0)
    opt = lambda a: None if a is None else to_dev(a, d)
    got = tl.kv_write_norm(kd, vd, to_dev(slots, d), kc, vc, k_scale=ks, v_scale=vs, q=qd, q_weight=opt(wq) if Hq else None,
                           k_weight=opt(wk), eps=eps, positions=to_dev(positions if axes > 1 else positions[0], d) if rot else None,
                           cos_sin=opt(cs), axis_of=opt(axis_of) if rot else None)
    torch.cuda.synchronize()

    def want(a, w):
        """The rows, and what f32 leaves open of each: the sum of squares has D / 16 + 4 roundings, the root, the quotient
        and two products one each; a turned pair's two products and their sum 3 of the pair's sizes."""
        y = ref.normed(a, w, eps)
        size = np.abs(y)
        if rot:
            h = rot // 2
            both = size[..., :h] + size[..., h:rot]
            size = np.concatenate([both, both, size[..., rot:]], -1)
            y = ref.turned(y, cs, positions, axis_of)
        return y, (D / 16 + 4 + 4 + 3) * F32_HALF * size
    if Hq:
        y, e = want(q, wq)
        assert (np.abs(f64(got) - y) <= BF16_HALF * np.abs(y) + 1.01 * e).all()
    else:
        assert got is None
    y, e = want(k, wk)
    served = (slots >= 0) & (slots < pages * block)
    es = 1 if e4m3 else 2
    rk, rv = bits(kc), bits(vc)
    k_at, v_at = (spec.offsets(c, es, block, D) for c in "kv")
    wv = np.full_like(rv, 0x5A if e4m3 else 0x5A5A)
    touched = np.zeros(rk.reshape(pages, H, -1).shape, dtype=bool)
    sk = ks.cpu().numpy() if e4m3 else None
    wvs = np.full((pages, H, block), -3.0, np.float32)
    untouched_scale = np.ones((pages, H, block), dtype=bool)
    bits_v = bits(vd)
    for t in np.flatnonzero(served):
        page, i = divmod(int(slots[t]), block)
        touched[page][:, k_at[i]] = True
        row = rk.reshape(pages, H, -1)[page][:, k_at[i]]
        if e4m3:
            top, et = np.abs(y[t]).max(-1), e[t].max(-1)
            scale = sk[page, :, i].astype(np.float64)
            assert (np.abs(scale - top / 448) <= 2 * F32_HALF * top / 448 + et / 448).all()
            # half a step of 3 mantissa bits, or of the smallest numbers' spacing
            miss = np.abs(spec.e4m3_value(row) * scale[:, None] - y[t])
            assert (miss <= (2.0 ** -4 + 2 * F32_HALF) * np.abs(y[t]) + 2 * e[t] + (2.0 ** -10 + F32_HALF) * scale[:, None]).all()
            assert (row[top == 0] == 0).all()
            sv = (np.abs(v[t]).max(-1).astype(np.float32) / np.float32(448))
            wvs[page, :, i], untouched_scale[page, :, i] = sv, False
            with np.errstate(invalid="ignore", divide="ignore"):
                code = spec.e4m3_code(np.where(sv[:, None] > 0, v[t].astype(np.float32) / sv[:, None], np.float32(0)))
            wv.reshape(pages, H, -1)[page][:, v_at[i]] = code
        else:
            value = (row.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
            assert (np.abs(value - y[t]) <= BF16_HALF * np.abs(y[t]) + 1.01 * e[t]).all()
            wv.reshape(pages, H, -1)[page][:, v_at[i]] = bits_v[t]
    np.testing.assert_array_equal(rv, wv)
    assert (rk.reshape(pages, H, -1)[~touched] == (0x5A if e4m3 else 0x5A5A)).all()
    if e4m3:
        np.testing.assert_array_equal(vs.cpu().numpy(), wvs)
        assert (sk[untouched_scale] == -3.0).all()


def test_kv_write_norm_without_norm_effect_is_kv_write(tl, torch):
    """Heads whose mean square is 1 - eps and weights of one: the rows of kv_write, up to the norm's roundings."""
    announce("kv_write_norm beside kv_write")
    d, T, H, D = dev(), 40, 2, 128
    rng = np.random.default_rng(3)
    x = np.where(rng.random((T, 3 * H, D)) < 0.5, -1.0, 1.0)
    xd = bf16_dev(x, d)
    cs = f32_dev(rng.uniform(-1, 1, (512, D)), d)
    slots, pos = to_dev(rng.permutation(64)[:T].astype(np.int64), d), to_dev(rng.integers(0, 512, T).astype(np.int32), d)
    a, b = (tl.kv_cache(4, H, 16, D, device=d) for _ in "ab")
    qa = tl.kv_write(xd[:, H:2 * H], xd[:, 2 * H:], slots, *a, q=xd[:, :H], positions=pos, cos_sin=cs)
    qb = tl.kv_write_norm(xd[:, H:2 * H], xd[:, 2 * H:], slots, *b, q=xd[:, :H], positions=pos, cos_sin=cs, eps=0.0)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(qa), bits(qb))
    for x, y in zip(a[:2], b[:2]):
        np.testing.assert_array_equal(bits(x), bits(y))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,Hq,D,rot,axes,gated,T", [(1, 8, 256, 64, 5, True, 8200), (2, 9, 64, 64, 1, False, 29300), (3, 33, 128, 32, 3, True, 4097)])
def test_kv_write_norm_of_a_prompt(tl, torch, H, Hq, D, rot, axes, gated, T, e4m3):
    """Thousands of tokens in one call: the same bits as the call cut into short ones, whose values the other tests
    check."""
    announce(f"kv_write_norm of a prompt T={T} H={H} Hq={Hq} D={D} e4m3={e4m3}")
    d, rng = dev(), np.random.default_rng(D)
    assert T * Hq >= 4096 * (256 // (D // 16)) > 1000 * Hq
    wide = 2 * D if gated else D
    x = torch.empty((T, Hq * wide + 2 * H * D + 8), dtype=torch.bfloat16, device=d).normal_(generator=torch.Generator(d).manual_seed(7))
    q = x[:, :Hq * wide].unflatten(1, (Hq, wide))[..., :D]
    k, v = (x[:, Hq * wide + i * H * D:][:, :H * D].unflatten(1, (H, D)) for i in (0, 1))
    wq, wk = (f32_dev(rng.standard_normal(D), d) for _ in "qk")
    pages = T // 64 + 2
    slots = rng.permutation(pages * 64)[:T].astype(np.int64)
    slots[rng.random(T) < 0.05] = -1
    slots = to_dev(slots, d)
    positions = to_dev(rng.integers(0, 4096, (axes, T)).astype(np.int32), d)
    axis_of = to_dev(rng.integers(0, axes, rot // 2).astype(np.int32), d) if axes > 1 else None
    cs = f32_dev(rng.uniform(-1, 1, (4096, rot)), d)
    caches, queries = [], []
    for cut in (T, 1000):
        kc, vc, ks, vs = tl.kv_cache(pages, H, 64, D, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device=d)
        for c in (kc, vc):
            c.view(torch.uint8).fill_(0x5A)
        if e4m3:
            ks.fill_(-3.0)
            vs.fill_(-3.0)
        qs = []
        for lo in range(0, T, cut):
            at = slice(lo, min(lo + cut, T))
            pos = positions[:, at].contiguous() if axes > 1 else positions[0, at]
            qs.append(tl.kv_write_norm(k[at], v[at], slots[at], kc, vc, k_scale=ks, v_scale=vs, q=q[at], q_weight=wq, k_weight=wk,
                                       positions=pos, cos_sin=cs, axis_of=axis_of))
        queries.append(torch.cat(qs))
        caches.append([c for c in (kc, vc, ks, vs) if c is not None])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(*(bits(y) for y in queries))
    assert torch.isfinite(queries[0].float()).all()
    for a, b in zip(*caches):
        np.testing.assert_array_equal(bits(a), bits(b))


# --------------------------------------------------------------------------- steps of requests with states
class Step:
    """Requests of these lengths: starts, lengths after the step, rows of states; tokens behind the last one."""

    def __init__(self, lens, rng, behind=3, unserved=True, trees=False):
        self.lens, R = lens, len(lens)
        self.q_start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.T = int(self.q_start[-1]) + behind
        ctx = rng.integers(1, 1000, R)
        ctx[rng.random(R) < 0.3] = 0                                   # these have just begun
        self.kv_lens = (ctx + lens).astype(np.int32)
        self.states = R + 3
        self.slots = rng.permutation(self.states)[:R].astype(np.int32)
        if unserved and R > 3:
            self.kv_lens[1], self.slots[2], self.slots[3] = 0, -1, self.states
        self.mask = None
        if trees:
            words = []
            for n in map(int, lens):
                m = []
                for i in range(n):
                    p = i - 1 if rng.random() < 0.5 else int(rng.random() * i)
                    m.append((m[p] if i and rng.random() < 0.95 else 0) | 1 << i)    # now and then another root
                    if rng.random() < 0.1 and i < 63:
                        m[i] |= 1 << int(rng.integers(i + 1, 64))                    # a bit past its own says nothing
                words += m if n <= 64 else [0] * int(n)
            self.mask = np.array(words + [0] * behind, dtype=np.uint64)

    def dev(self, d):
        return [to_dev(a, d) for a in (self.q_start, self.kv_lens, self.slots)]

    def mask_dev(self, d):
        return None if self.mask is None else to_dev(self.mask.view(np.int64), d)


LENGTHS = [[1], [0, 3, 0], [1, 2, 3, 4, 1], [16, 15, 17, 1, 0, 33], [64, 63, 65, 1, 31, 32, 128], [130, 2, 200, 0, 7]]


@pytest.mark.parametrize("trees", [False, True])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("taps,C,heads,dim,bias", [(4, 640, 2, 128, False), (2, 8, 0, 128, True), (3, 2200, 3, 64, True), (4, 512, 2, 256, True)])
def test_short_conv(tl, torch, taps, C, heads, dim, bias, lens, trees):
    announce(f"short_conv taps={taps} C={C} heads={heads}x{dim} lens={lens} trees={trees}")
    d, rng = dev(), np.random.default_rng(sum(lens) + C + taps + trees)
    s = Step(np.array(lens), rng, trees=trees)
    x = spec.bf16(rng.standard_normal((s.T, C + 16)))
    x[rng.random(s.T) < 0.05] = 0.0
    w = rng.standard_normal((C, taps)).astype(np.float32)
    b = rng.standard_normal(C).astype(np.float32) if bias else None
    state = spec.bf16(rng.standard_normal((s.states, taps - 1, C)))
    stated, xd = bf16_dev(state, d), bf16_dev(x, d)
    if len(lens) > 3:                                     # what lies in a row that nobody reads does not matter
        free = np.setdiff1d(np.arange(s.states), s.slots)
        stated[int(free[0])] = float("nan")
    out = torch.full((s.T, C + 8), -7.0, dtype=torch.bfloat16, device=d)
    before = stated.clone()
    eps = 1e-6
    tl.short_conv(xd[:, 8:8 + C], to_dev(w, d), *s.dev(d), stated, bias=None if b is None else to_dev(b, d),
                  tree_mask=s.mask_dev(d), norm_heads=heads, norm_dim=dim, eps=eps, out=out[:, :C])
    torch.cuda.synchronize()
    want, after, err = ref.short_conv(x[:, 8:8 + C], w.astype(np.float64), b, s.q_start, s.kv_lens, s.slots, f64(before),
                                      s.mask, heads, dim, eps, np.full((s.T, C), -7.0))
    got = f64(out[:, :C])
    assert (np.abs(got - want) <= BF16_HALF * np.abs(want) + 1.01 * F32_HALF * err).all()
    assert (got[s.q_start[-1]:] == -7.0).all() and (f64(out[:, C:]) == -7.0).all()
    np.testing.assert_array_equal(f64(stated), after)


@pytest.mark.parametrize("run,C", [(16, 8192), (32, 12288), (64, 32768)])
@pytest.mark.parametrize("taps", [2, 3, 4])
def test_short_conv_long_runs(tl, torch, taps, run, C):
    """Enough tokens and channels for runs of this many tokens, with requests that end inside a run, and trees among them."""
    announce(f"short_conv runs of {run} taps={taps}")
    d, rng = dev(), np.random.default_rng(taps)
    s = Step(np.array([1500, 1, 0, 63, 64, 65, 700, 3] + [20] * 70), rng, trees=taps == 3)
    assert s.T // run * (C // 2048) >= 512 and (run == 64 or s.T // (2 * run) * (C // 2048) < 512)
    heads = C // 128                                                   # half of the channels
    x = spec.bf16(rng.standard_normal((s.T, 64)))
    w = rng.standard_normal((64, taps)).astype(np.float32)
    state = spec.bf16(rng.standard_normal((s.states, taps - 1, 64)))
    wide = lambda a: a.repeat(*([1] * (a.dim() - 1)), C // 64)         # the same 64 channels again and again
    stated = wide(bf16_dev(state, d))
    out = torch.full((s.T, C), -7.0, dtype=torch.bfloat16, device=d)
    tl.short_conv(wide(bf16_dev(x, d)), to_dev(w, d).repeat(C // 64, 1), *s.dev(d), stated, tree_mask=s.mask_dev(d), norm_heads=heads,
                  norm_dim=64, out=out)
    torch.cuda.synchronize()
    want, after, err = ref.short_conv(x, w.astype(np.float64), None, s.q_start, s.kv_lens, s.slots, state, s.mask, 1, 64, 1e-6,
                                      np.full((s.T, 64), -7.0))
    plain, _, e0 = ref.short_conv(x, w.astype(np.float64), None, s.q_start, s.kv_lens, s.slots, state, s.mask, 0, 64, 1e-6,
                                  np.full((s.T, 64), -7.0))
    got = f64(out).reshape(s.T, C // 64, 64)
    tol = lambda v, e: BF16_HALF * np.abs(v) + 1.01 * F32_HALF * e
    assert (np.abs(got[:, :heads] - want[:, None]) <= tol(want, err)[:, None]).all()
    assert (np.abs(got[:, heads:] - plain[:, None]) <= tol(plain, e0)[:, None]).all()
    np.testing.assert_array_equal(f64(stated).reshape(s.states, taps - 1, C // 64, 64), np.repeat(after[:, :, None], C // 64, 2))


def _delta_inputs(s, Hk, G, Dk, Dv, rng, raw, d, decay=0.3):
    T, Hv = s.T, Hk * G
    unit = lambda n: (lambda y: y / np.sqrt((y * y).sum(-1, keepdims=True)))(rng.standard_normal((T, n, Dk)) + 0.4)
    y = np.concatenate([unit(Hk).reshape(T, -1), unit(Hk).reshape(T, -1), rng.standard_normal((T, Hv * Dv)),
                        np.zeros((T, 8))], 1)
    y = spec.bf16(y)
    yd = bf16_dev(y, d)
    cols = lambda a, lo, n, w: a[:, lo:lo + n * w].reshape(T, n, w)
    q, k, v = (cols(y, lo, n, w) for lo, n, w in ((0, Hk, Dk), (Hk * Dk, Hk, Dk), (2 * Hk * Dk, Hv, Dv)))
    qd, kd, vd = (yd[:, lo:lo + n * w].unflatten(1, (n, w)) for lo, n, w in ((0, Hk, Dk), (Hk * Dk, Hk, Dk), (2 * Hk * Dk, Hv, Dv)))
    ab = rng.standard_normal((T, 2 * Hv + 1)).astype(np.float32)
    log, bias = None, None
    if raw:
        log, bias = (rng.uniform(-2, 1, Hv).astype(np.float32) for _ in "ab")
        g, b = ref.gates(ab[:, :Hv].astype(np.float64), ab[:, Hv:-1].astype(np.float64), log.astype(np.float64), bias.astype(np.float64))
    else:
        ab[:, :Hv] = -decay * np.exp(ab[:, :Hv])
        ab[:, Hv:-1] = 1 / (1 + np.exp(-ab[:, Hv:-1]))
        g, b = ab[:, :Hv].astype(np.float64), ab[:, Hv:-1].astype(np.float64)
    abd = to_dev(ab, d)
    state = (0.3 * rng.standard_normal((s.states, Hv, Dk, Dv))).astype(np.float32)
    opt = lambda a: None if a is None else to_dev(a, d)
    return (q, k, v, g, b), (qd, kd, vd, abd[:, :Hv], abd[:, Hv:-1]), dict(a_log=opt(log), dt_bias=opt(bias)), state


def _check_delta(got, got_state, want, want_state, size, before, tokens):
    """Outputs and states against the definition's; states that nobody advanced are bit for bit what they were."""
    # below f32's smallest normal number, 2^-126, relative bounds end: a state that has decayed to nothing gives sums of
    # up to 128 + 64 terms (and as many products behind each u) that may each have been flushed
    tol = BF16_HALF * np.abs(want) + PARTS * size + STATE_TOL * size + 2.0 ** (-126 + 8)
    worst = np.unravel_index(np.argmax(np.abs(got - want) / tol), got.shape)
    assert (np.abs(got - want) <= tol).all(), (worst, got[worst], want[worst], tol[worst])
    assert (got[tokens:] == -7.0).all()
    for row in range(len(before)):
        if np.array_equal(want_state[row], before[row].astype(np.float64), equal_nan=True):
            np.testing.assert_array_equal(got_state[row], before[row])
        else:
            miss = np.linalg.norm(got_state[row].astype(np.float64) - want_state[row])
            assert miss <= STATE_TOL * np.linalg.norm(want_state[row]), (row, miss / np.linalg.norm(want_state[row]))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("Hk,G,Dk,Dv,raw", [(1, 1, 64, 16, False), (2, 3, 128, 128, True), (3, 1, 64, 80, True), (1, 4, 128, 48, False)])
def test_delta_rule(tl, torch, Hk, G, Dk, Dv, raw, lens, form):
    announce(f"delta_rule {form} Hk={Hk} G={G} Dk={Dk} Dv={Dv} raw={raw} lens={lens}")
    d, rng = dev(), np.random.default_rng(sum(lens) + Dk + Dv + G)
    s = Step(np.array(lens), rng, trees="trees" in form)
    plain, given, gates, state = _delta_inputs(s, Hk, G, Dk, Dv, rng, raw, d)
    free = np.setdiff1d(np.arange(s.states), s.slots)
    state[free[0]] = np.nan                               # a row that nobody reads
    for r in range(len(lens)):                            # a request that has just begun does not read its row either
        if s.kv_lens[r] <= lens[r] and 0 <= s.slots[r] < s.states and 0 < s.kv_lens[r]:
            state[s.slots[r]] = np.inf
    stated = to_dev(state, d)
    out = torch.full((s.T, Hk * G, Dv), -7.0, dtype=torch.bfloat16, device=d)
    tl.delta_rule(*given, *s.dev(d), stated, **gates, tree_mask=s.mask_dev(d), max_nodes=FORMS[form], out=out)
    torch.cuda.synchronize()
    assert tl.last_kernel_name() == KERNEL.get(form, "delta_scan")
    want, after, size = ref.delta_rule(*plain, s.q_start, s.kv_lens, s.slots, state.astype(np.float64), s.mask, Dk ** -0.5,
                                       np.full((s.T, Hk * G, Dv), -7.0))
    _check_delta(f64(out), stated.cpu().numpy(), want, after, size, state, s.q_start[-1])


@pytest.mark.parametrize("op", ["conv", *FORMS, "commit"])
@pytest.mark.parametrize("R", [64, 65, 300, 513])
def test_many_requests(tl, torch, R, op):
    """More requests than a wave's lanes, than a workgroup's, than twice that; and more columns than a tree's workgroup has."""
    announce(f"{op} of {R} requests")
    d, rng = dev(), np.random.default_rng(R)
    lens = rng.integers(0, 4, R)
    lens[[0, R // 2, R - 1]] = 66, 20, 9
    s = Step(lens, rng, trees="trees" in op or op == "commit")
    Hk, G, Dk, Dv = 1, 2, 64, 144
    plain, given, _, state = _delta_inputs(s, Hk, G, Dk, Dv, rng, False, d)
    stated = to_dev(state, d)
    if op == "conv":
        x, w = spec.bf16(rng.standard_normal((s.T, 64))), rng.standard_normal((64, 4)).astype(np.float32)
        conv = spec.bf16(rng.standard_normal((s.states, 3, 64)))
        convd = bf16_dev(conv, d)
        got = f64(tl.short_conv(bf16_dev(x, d), to_dev(w, d), *s.dev(d), convd))
        want, after, err = ref.short_conv(x, w.astype(np.float64), None, s.q_start, s.kv_lens, s.slots, conv, None, 0, 64, 1e-6,
                                          np.zeros((s.T, 64)))
        n = s.q_start[-1]
        assert (np.abs(got - want)[:n] <= (BF16_HALF * np.abs(want) + 1.01 * F32_HALF * err)[:n]).all()
        np.testing.assert_array_equal(f64(convd), after)
        return
    if op == "commit":
        path = np.sort(rng.random((R, 70)).argsort(1)[:, :4] % np.maximum(lens, 1)[:, None], 1).astype(np.int32)
        accepted = rng.integers(0, 5, R).astype(np.int32)
        tl.delta_commit(to_dev(accepted, d), to_dev(path, d), *s.dev(d), *given[1:], stated)
        torch.cuda.synchronize()
        want, _ = ref.delta_commit(accepted, path, s.q_start, s.kv_lens, s.slots, *plain[1:], state.astype(np.float64),
                                   np.zeros((s.T, 8)), np.zeros((s.states, 3, 8)))
        got = stated.cpu().numpy()
        for row in range(s.states):
            assert np.linalg.norm(got[row] - want[row]) <= STATE_TOL * np.linalg.norm(want[row]), row
        return
    out = torch.full((s.T, Hk * G, Dv), -7.0, dtype=torch.bfloat16, device=d)
    tl.delta_rule(*given, *s.dev(d), stated, tree_mask=s.mask_dev(d),
                  max_nodes=FORMS[op], out=out)
    torch.cuda.synchronize()
    want, after, size = ref.delta_rule(*plain, s.q_start, s.kv_lens, s.slots, state.astype(np.float64), s.mask, Dk ** -0.5,
                                       np.full((s.T, Hk * G, Dv), -7.0))
    _check_delta(f64(out), stated.cpu().numpy(), want, after, size, state, s.q_start[-1])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kind", ["resets", "far", "same keys", "no steps", "kept"])
def test_delta_rule_extremes(tl, torch, kind, form):
    """Decays of exp(-inf) and far below any exponent between ordinary ones, the same key again and again with a step
    of one (the solved system at its worst), steps of zero, and no decay at all."""
    announce(f"delta_rule extremes {kind} {form}")
    d, rng = dev(), np.random.default_rng(11)
    lens = [64, 40, 1] if "trees" in form or form == "one chunk" else [150, 64, 1]
    s = Step(np.array(lens), rng, trees="trees" in form)
    (q, k, v, g, b), (qd, kd, vd, ad, bd), _, state = _delta_inputs(s, 2, 2, 64, 32, rng, False, d)
    if kind == "resets":
        g[::7] = -np.inf
    elif kind == "far":
        g[::5] = rng.uniform(-3000, -80, g[::5].shape)
    elif kind == "same keys":
        k[:] = k[:1]
        b[:], g[:] = 1.0, -0.01
    elif kind == "no steps":
        b[:] = 0.0
    else:
        g[:] = 0.0
    g, b = g.astype(np.float32), b.astype(np.float32)
    stated = to_dev(state, d)
    out = torch.full((s.T, 4, 32), -7.0, dtype=torch.bfloat16, device=d)
    tl.delta_rule(qd, bf16_dev(k, d), vd, to_dev(g, d), to_dev(b, d), *s.dev(d), stated, tree_mask=s.mask_dev(d),
                  max_nodes=FORMS[form], out=out)
    torch.cuda.synchronize()
    want, after, size = ref.delta_rule(q, k, v, g.astype(np.float64), b.astype(np.float64), s.q_start, s.kv_lens, s.slots,
                                       state.astype(np.float64), s.mask, 0.125, np.full((s.T, 4, 32), -7.0))
    _check_delta(f64(out), stated.cpu().numpy(), want, after, size, state, s.q_start[-1])


def test_delta_rule_not_finite_stays_where_it_is(tl, torch):
    """NaN and infinities in one request's rows, in rows behind the last one and in a tree's other branch do not reach
    other requests or other branches."""
    announce("delta_rule with NaN and infinities beside")
    d, rng = dev(), np.random.default_rng(5)
    for form in FORMS:
        s = Step(np.array([20, 40, 33]), rng, behind=64, trees="trees" in form)
        if "trees" in form:                               # request 1: two chains from the root, 1..19 and 20..39
            first = int(s.q_start[1])
            for i in range(40):
                s.mask[first + i] = (1 << i + 1) - 1 if i < 20 else 1 | ((1 << i + 1) - 1 >> 20 << 20)
        plain, given, _, state = _delta_inputs(s, 1, 2, 128, 32, rng, False, d)
        bad = np.zeros(s.T, dtype=bool)
        bad[:20] = bad[93:] = True
        if "trees" in form:
            bad[20 + 20:20 + 40] = True
        rows = torch.from_numpy(bad).to(d)
        q, k, v, a, b = (x.clone() for x in given)
        for x, fill in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (a, float("nan")), (b, float("inf"))):
            x[rows] = fill
        stated = to_dev(state, d)
        out = torch.full((s.T, 2, 32), -7.0, dtype=torch.bfloat16, device=d)
        tl.delta_rule(q, k, v, a, b, *s.dev(d), stated, tree_mask=s.mask_dev(d), max_nodes=FORMS[form], out=out)
        torch.cuda.synchronize()
        want, after, size = ref.delta_rule(*plain, s.q_start, s.kv_lens, s.slots, state.astype(np.float64), s.mask, 128 ** -0.5,
                                           np.full((s.T, 2, 32), -7.0))
        if "trees" in form:                               # no state is touched, whatever the tokens held
            np.testing.assert_array_equal(stated.cpu().numpy(), state)
        else:
            assert np.isnan(stated.cpu().numpy()[s.slots[0]]).all() == (s.kv_lens[0] > 0 and s.slots[0] >= 0)
        good = ~bad[:93]
        tol = (BF16_HALF * np.abs(want) + (PARTS + STATE_TOL) * size)[:93][good]
        assert (np.abs(f64(out)[:93][good] - want[:93][good]) <= tol).all(), form
        assert (f64(out)[93:] == -7.0).all()
        for r in (1, 2):
            row = s.slots[r]
            assert np.linalg.norm(stated.cpu().numpy()[row] - after[row]) <= STATE_TOL * np.linalg.norm(after[row]), (form, r)


@pytest.mark.parametrize("op", ["conv", *FORMS, "commit"])
@pytest.mark.parametrize("starts", [[0, 5, 3, 9], [-1, 2, 3, 9], [0, 2, 3, 10], [9, 0, 0, 0], [0, 0, 12, 9]], ids=str)
def test_starts_that_fall_write_nothing(tl, torch, starts, op):
    announce(f"starts {starts} {op}")
    d, rng = dev(), np.random.default_rng(2)
    s = Step(np.array([3, 3, 3]), rng, behind=0, trees="trees" in op or op == "commit")
    s.q_start = np.array(starts, dtype=np.int32)
    _, (q, k, v, a, b), _, state = _delta_inputs(s, 1, 1, 64, 16, rng, False, d)
    stated = to_dev(state, d)
    conv = bf16_dev(rng.standard_normal((s.states, 3, 64)), d)
    before = stated.clone(), conv.clone()
    x = bf16_dev(rng.standard_normal((9, 64)), d)
    if op == "conv":
        out = torch.full((9, 64), -7.0, dtype=torch.bfloat16, device=d)
        tl.short_conv(x, f32_dev(rng.standard_normal((64, 4)), d), *s.dev(d), conv, out=out)
    elif op == "commit":
        out = torch.full((1,), -7.0, device=d)
        tl.delta_commit(to_dev(np.array([1, 2, 3], np.int32), d), to_dev(np.array([[0, 1, 2]] * 3, np.int32), d), *s.dev(d), k, v,
                        a, b, stated, x=x, conv_state=conv)
    else:
        out = torch.full((9, 1, 16), -7.0, dtype=torch.bfloat16, device=d)
        tl.delta_rule(q, k, v, a, b, *s.dev(d), stated, tree_mask=s.mask_dev(d), max_nodes=FORMS[op], out=out)
    torch.cuda.synchronize()
    assert (out == -7.0).all()
    assert torch.equal(stated, before[0]) and torch.equal(conv, before[1])


@pytest.mark.parametrize("what", ["q", "k", "v", "a", "b"])
@pytest.mark.parametrize("form", FORMS)
def test_delta_rule_not_finite_later_tokens_only(tl, torch, form, what):
    """A token whose rows are not finite spoils its own result and those of the tokens that see it, and no other's."""
    announce(f"delta_rule with a {what} that is not finite, {form}")
    d, rng = dev(), np.random.default_rng(6)
    short = "trees" in form or form == "one chunk"
    s = Step(np.array([50 if short else 150]), rng, trees="trees" in form)
    plain, given, _, state = _delta_inputs(s, 1, 2, 64, 32, rng, False, d)
    at = 21 if short else 90
    given = [x.clone() for x in given]
    j = "qkvab".index(what)
    given[j][at, 0] = float("nan") if what in "qa" else float("inf")
    if what == "v":
        given[j][at, 0, 3:] = given[j][at + 1, 0, 3:]      # columns 0 to 2 of head 0 only
    stated = to_dev(state, d)
    out = tl.delta_rule(*given, *s.dev(d), stated, tree_mask=s.mask_dev(d), max_nodes=FORMS[form])
    torch.cuda.synchronize()
    v = plain[2].copy()
    if what == "v":
        v[at, 0, 3:] = v[at + 1, 0, 3:]
    want, after, size = ref.delta_rule(plain[0], plain[1], v, *plain[3:], s.q_start, s.kv_lens, s.slots, state.astype(np.float64),
                                       s.mask, 0.125, np.zeros((s.T, 2, 32)))
    n = int(s.lens[0])
    sees = np.array([at in line for line in ref.lines(n, "trees" in form, s.mask)])
    spoilt = np.zeros((n, 2, 32), dtype=bool)
    heads, cols = (slice(None), slice(None)) if what in "qk" else (0, slice(3)) if what == "v" else (0, slice(None))
    spoilt[(at if what == "q" else sees), heads, cols] = True
    got = f64(out)[:n]
    assert not np.isfinite(got[spoilt]).any()
    tol = BF16_HALF * np.abs(want[:n]) + (PARTS + STATE_TOL) * size[:n]
    assert (np.abs(got - want[:n])[~spoilt] <= tol[~spoilt]).all()
    row, S = s.slots[0], stated.cpu().numpy()
    if "trees" in form:
        np.testing.assert_array_equal(S, state)
    elif what == "q":
        assert np.linalg.norm(S[row] - after[row]) <= STATE_TOL * np.linalg.norm(after[row])
    else:
        lost = np.zeros((2, 64, 32), dtype=bool)
        lost[heads, :, cols] = True
        assert not np.isfinite(S[row][lost]).any()
        assert np.linalg.norm((S[row] - after[row])[~lost]) <= STATE_TOL * np.linalg.norm(after[row][~lost])


# --------------------------------------------------------------------------- commit
@pytest.mark.parametrize("L,Hk,G,Dk,Dv,taps,width,raw", [(1, 1, 1, 64, 16, 4, 64, False), (3, 2, 3, 128, 128, 4, 9, True),
                                                         (2, 1, 2, 128, 80, 2, 64, True), (2, 3, 1, 64, 32, 3, 5, False)])
def test_delta_commit(tl, torch, L, Hk, G, Dk, Dv, taps, width, raw):
    announce(f"delta_commit L={L} Hk={Hk} G={G} Dk={Dk} Dv={Dv} taps={taps} width={width} raw={raw}")
    d, rng = dev(), np.random.default_rng(L + Dk + Dv)
    lens = [5, 3, 2, 4, 64, 1, 0, 65, 17, 30]
    s = Step(np.array(lens), rng, trees=True)
    R, C = len(lens), 2 * Hk * Dk + Hk * G * Dv
    layers = [_delta_inputs(s, Hk, G, Dk, Dv, rng, raw, d) for _ in range(L)]
    x = spec.bf16(rng.standard_normal((L, s.T, C)))
    conv = spec.bf16(rng.standard_normal((L, s.states, taps - 1, C)))
    state = np.stack([p[3] for p in layers])
    path = np.full((R, width), -1, np.int32)
    accepted = np.zeros(R, np.int32)
    for r, n in enumerate(lens):
        count = int(rng.integers(0, min(max(n, 1), width))) + 1
        nodes = np.sort(rng.permutation(max(n, count))[:count])
        path[r, :count], accepted[r] = nodes, count
    accepted[5], accepted[9] = 0, 70                      # nothing accepted; more than the path and the request have
    if width > 8:
        path[8, 1], path[4, 2] = -3, 1 << 30              # entries that name no token
    stated, convd = to_dev(state, d), bf16_dev(conv, d)
    stack = lambda j: torch.stack([p[1][j] for p in layers])
    log = dict(a_log=torch.stack([p[2]["a_log"] for p in layers]), dt_bias=torch.stack([p[2]["dt_bias"] for p in layers])) if raw else {}
    tl.delta_commit(to_dev(accepted, d), to_dev(path, d), *s.dev(d), stack(1), stack(2), stack(3), stack(4), stated, **log,
                    x=bf16_dev(x, d), conv_state=convd)
    torch.cuda.synchronize()
    got = stated.cpu().numpy()
    for layer in range(L):
        _, k, v, g, b = layers[layer][0]
        want, want_conv = ref.delta_commit(accepted, path, s.q_start, s.kv_lens, s.slots, k, v, g, b,
                                           state[layer].astype(np.float64), x[layer], conv[layer])
        np.testing.assert_array_equal(f64(convd[layer]), want_conv)
        for row in range(s.states):
            if np.array_equal(want[row], state[layer, row].astype(np.float64)):
                np.testing.assert_array_equal(got[layer, row], state[layer, row])
            else:
                assert np.linalg.norm(got[layer, row] - want[row]) <= STATE_TOL * np.linalg.norm(want[row])
    if L == 1:                                            # one layer without the leading dimension, and without x
        again = to_dev(state[0], d)
        tl.delta_commit(to_dev(accepted, d), to_dev(path, d), *s.dev(d), *(layers[0][1][j] for j in (1, 2, 3, 4)), again)
        torch.cuda.synchronize()
        assert torch.equal(again, stated[0])


def test_states_past_32_bits(tl, torch):
    """A row whose elements begin past 2^32 of the pool."""
    announce("states past 2^32 elements")
    d, rng = dev(), np.random.default_rng(8)
    s = Step(np.array([70, 3]), rng)
    Hk, G, Dk, Dv = 2, 2, 128, 128
    per = Hk * G * Dk * Dv
    states = (1 << 32) // per + 3
    plain, given, _, state = _delta_inputs(s, Hk, G, Dk, Dv, rng, False, d)
    pool = torch.empty((states, Hk * G, Dk, Dv), dtype=torch.float32, device=d)
    s.kv_lens = (np.array([70, 3]) + 5).astype(np.int32)
    small = np.array([1, 0], np.int32)
    s.slots = np.array([states - 1, states - 2], np.int32)
    for form in (1, 64, 1000):
        pool[states - 2:] = to_dev(state[:2], d)
        out = torch.full((s.T, Hk * G, Dv), -7.0, dtype=torch.bfloat16, device=d)
        tl.delta_rule(*given, *s.dev(d), pool, max_nodes=form, out=out)
        torch.cuda.synchronize()
        want, after, size = ref.delta_rule(*plain, s.q_start, s.kv_lens, small, state[:2].astype(np.float64), None, Dk ** -0.5,
                                           np.full((s.T, Hk * G, Dv), -7.0))
        _check_delta(f64(out), pool[states - 2:].cpu().numpy(), want, after, size, state[:2], 73)
    pool[states - 2:] = to_dev(state[:2], d)
    _, k, v, a, b = given
    tl.delta_commit(to_dev(np.array([0, 2], np.int32), d), to_dev(np.array([[0, 1]] * 2, np.int32), d), *s.dev(d), k, v, a, b, pool)
    torch.cuda.synchronize()
    want, _ = ref.delta_commit([0, 2], [[0, 1]] * 2, s.q_start, s.kv_lens, small, *plain[1:], state[:2].astype(np.float64),
                               np.zeros((s.T, 8)), np.zeros((2, 3, 8)))
    assert np.linalg.norm(pool[states - 2].cpu().numpy() - want[0]) <= STATE_TOL * np.linalg.norm(want[0])
    del pool
    torch.cuda.empty_cache()


# --------------------------------------------------------------------------- together
def test_a_step_captured_and_replayed(tl, torch):
    """Prompt chunk, then a tree step and its commit, captured in one graph on a side stream and replayed between eager
    work; every replay gives the eager result bit for bit."""
    announce("mixers captured and replayed")
    d, rng = dev(), np.random.default_rng(21)
    Hk, G, Dk, Dv, taps = 2, 2, 64, 64, 4
    C, Hv = 2 * Hk * Dk + Hk * G * Dv, Hk * G
    chain, tree = Step(np.array([130, 5, 64]), rng, unserved=False), Step(np.array([9, 64, 1]), rng, trees=True)
    tree.slots[:], tree.states = chain.slots, chain.states
    data = [(bf16_dev(rng.standard_normal((s.T, C)), d), f32_dev(rng.standard_normal((s.T, 2 * Hv)), d), s.dev(d), s.mask_dev(d))
            for s in (chain, tree)]
    w, log, bias = f32_dev(rng.standard_normal((C, taps)), d), f32_dev(rng.uniform(-2, 0, Hv), d), f32_dev(rng.uniform(-1, 1, Hv), d)
    state0, conv0 = f32_dev(rng.standard_normal((chain.states, Hv, Dk, Dv)), d), bf16_dev(rng.standard_normal((chain.states, taps - 1, C)), d)
    state, conv = state0.clone(), conv0.clone()
    accepted, path = to_dev(np.array([2, 3, 1], np.int32), d), to_dev(np.array([[0, 4, -1], [0, 1, 9], [0, -1, -1]], np.int32), d)
    ys = [torch.empty((s.T, C), dtype=torch.bfloat16, device=d) for s in (chain, tree)]
    outs = [torch.empty((s.T, Hv, Dv), dtype=torch.bfloat16, device=d) for s in (chain, tree)]
    work = torch.empty(max(tl.delta_rule_workspace_size(s.T, 3, Hk, G, Dk, 130, True) for s in (chain, tree)), dtype=torch.uint8, device=d)

    def step():
        state.copy_(state0)
        conv.copy_(conv0)
        for (x, ab, meta, mask), y, out in zip(data, ys, outs):
            tl.short_conv(x, w, *meta, conv, tree_mask=mask, norm_heads=2 * Hk, norm_dim=Dk, out=y)
            q, k, v = (part.unflatten(1, (-1, n)) for part, n in zip(y.split((Hk * Dk, Hk * Dk, Hv * Dv), 1), (Dk, Dk, Dv)))
            tl.delta_rule(q, k, v, ab[:, :Hv], ab[:, Hv:], *meta, state, a_log=log, dt_bias=bias, tree_mask=mask, max_nodes=130,
                          out=out, workspace=work)
        tl.delta_commit(accepted, path, *meta, k, v, ab[:, :Hv], ab[:, Hv:], state, a_log=log, dt_bias=bias, x=x, conv_state=conv)

    for t in ys + outs:
        t.fill_(0)
    step()
    torch.cuda.synchronize()
    kept = [t.clone() for t in (state, conv, *ys, *outs)]
    assert all(torch.isfinite(t.float()).all() for t in kept)
    side = torch.cuda.Stream(d)
    side.wait_stream(torch.cuda.current_stream(d))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream(d).wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for r in range(3):
        work.fill_(0xFF)                                  # NaN everywhere: nothing of it may be read before it is written
        for t in outs:
            t.fill_(0)
        for t in ys:
            t.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        announce(f"  replay {r}")
        for a, b in zip((state, conv, *ys, *outs), kept):
            assert torch.equal(a, b)
    # a chain given as a tree, committed whole, is the chain
    s = Step(np.array([30, 64, 7]), rng, behind=0)
    given = _delta_inputs(s, Hk, G, Dk, Dv, rng, False, d)[1]
    chain_state, tree_state = state0[:s.states].clone(), state0[:s.states].clone()
    as_tree = to_dev(np.array([(1 << i + 1) - 1 for n in s.lens for i in range(n)], dtype=np.uint64).view(np.int64), d)
    a = tl.delta_rule(*given, *s.dev(d), chain_state, max_nodes=64)
    b = tl.delta_rule(*given, *s.dev(d), tree_state, tree_mask=as_tree, max_nodes=64)
    parts_state = state0[:s.states].clone()
    c = tl.delta_rule(*given, *s.dev(d), parts_state, max_nodes=65)
    torch.cuda.synchronize()
    assert (parts_state - chain_state).norm() <= 2 * STATE_TOL * chain_state.norm()
    assert (c.double() - a.double()).norm() <= 2 * BF16_HALF * a.double().norm()
    assert torch.equal(a, b) and torch.equal(tree_state, state0[:s.states])
    tl.delta_commit(to_dev(s.lens.astype(np.int32), d), to_dev(np.tile(np.arange(64, dtype=np.int32), (3, 1)), d), *s.dev(d), *given[1:], tree_state)
    torch.cuda.synchronize()
    assert (tree_state - chain_state).norm() <= 2 * STATE_TOL * chain_state.norm()


def test_default_stream_order_and_other_streams(tl, torch):
    """Calls on a stream of their own see what that stream has written, without a synchronisation."""
    announce("mixers on another stream")
    d, rng = dev(), np.random.default_rng(4)
    s = Step(np.array([100, 80]), rng, behind=0, unserved=False)
    _, given, _, state = _delta_inputs(s, 1, 2, 128, 64, rng, False, d)
    want_state = to_dev(state, d)
    want = tl.delta_rule(*given, *s.dev(d), want_state, max_nodes=100)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(d)
    with torch.cuda.stream(side):
        got_state = torch.zeros_like(want_state)
        big = torch.ones(1 << 26, device=d)
        for _ in range(20):
            big.mul_(1.0001)                              # the stream is busy while the call is issued
        got_state.copy_(to_dev(state, d))
        got = tl.delta_rule(*given, *s.dev(d), got_state, max_nodes=100)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(got_state, want_state)
