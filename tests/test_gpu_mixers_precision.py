"""How exact the gated delta rule's outputs and states are: outputs whose large terms cancel, so that what is left would be
gone if an operand had lost its last bits, in every form of the operator."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.mixers as ref
import oracle.speculative as spec
from gpu_common import announce, to_dev
from test_gpu_mixers import BF16_HALF, F32_HALF, FORMS, KERNEL, bf16_dev, dev, f64, tl, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

X, Y = 1 + 2.0 ** -9 + 2.0 ** -17, 1 + 2.0 ** -9    # X takes 18 bits: three parts of 8


@pytest.mark.parametrize("what", ["state", "weights", "updates", "both"])
@pytest.mark.parametrize("at", [(0, 1, 2), (1, 20, 21), (5, 40, 63), (30, 33, 47), (64 + 3, 64 + 30, 64 + 50), (2, 100, 130)], ids=str)
@pytest.mark.parametrize("Dk", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_what_cancellation_leaves(tl, torch, form, Dk, at, what):  # noqa: F811
    """Token at[2] reads X - Y (or products of such numbers) as the difference of two terms of about 1: of the state from
    before the step, of the weights q k, of the updates u, or of the products of weights and updates.  f32 holds every
    operand, and each term is rounded once or twice and added in f32 (2^-24 of 2.02 each, at most 8 of them): the
    remainder of 2^-17 or 2^-18 is good to a quarter at the worst.  Without an operand's last 8 bits it is 0."""
    if at[2] >= 64 and (form == "one chunk" or form == "trees"):
        at = tuple(i % 64 for i in at)
        at = tuple(sorted(at))
    if len(set(at)) < 3:
        at = (at[0], at[0] + 1, at[0] + 2)
    announce(f"cancellation of {what} in {form}, Dk={Dk}, tokens {at}")
    d, n, Dv = dev(), at[2] + 5, 48
    i0, i1, i2 = at
    q, k, v = np.zeros((n, 1, Dk)), np.zeros((n, 1, Dk)), np.zeros((n, 1, Dv))
    g, b = np.zeros((n, 1), np.float32), np.zeros((n, 1), np.float32)
    state = np.zeros((1, 1, Dk, Dv), np.float32)
    cols = 2.0 ** (np.arange(Dv) % 5 - 2)
    left = 2.0 ** -17
    if what == "state":
        q[i2, 0, [3, 40]] = 1.0
        state[0, 0, 3], state[0, 0, 40] = X * cols, -Y * cols
    else:
        v[i0, 0], v[i1, 0] = cols, -cols
        b[[i0, i1]] = 1.0
        e = [1, 9, 33, 50, 62]                             # elements of keys that are not 0
        if what == "weights":                              # q k = X and Y, the two keys orthogonal
            q[i2, 0, e[:3]] = 1, 2.0 ** -4, 2.0 ** -8
            k[i0, 0, e] = 1, 2.0 ** -5, 2.0 ** -9, 1, 2.0 ** -5
            k[i1, 0, e] = 1, 2.0 ** -5, 0, -1, -2.0 ** -5
        elif what == "updates":                            # u = X and -Y
            q[i2, 0, e[:2]] = 1.0
            k[i0, 0, e[0]] = k[i1, 0, e[1]] = 1.0
            b[i0], b[i1] = X, Y
        else:                                              # (1 + 2^-9)^2 - (1 + 2^-8)
            q[i2, 0, e[:2]] = 1, 2.0 ** -4
            k[i0, 0, e[:4]] = 1, 2.0 ** -5, 0, 1
            k[i1, 0, e[:4]] = 1, 0, 0, -1
            b[i0], b[i1] = Y, 1 + 2.0 ** -8
            left = 2.0 ** -18
    want = np.zeros((n, 1, Dv))
    want[i2, 0] = left * cols
    mask = None
    if "trees" in form:
        words = np.array([(2 << i % 64) - 1 for i in range(n)], dtype=np.uint64) if n <= 64 else np.zeros(n, np.uint64)
        mask = to_dev(words.view(np.int64), d)
    meta = [to_dev(np.array(x, np.int32), d) for x in ([0, n], [n + 9], [0])]
    out = tl.delta_rule(bf16_dev(q, d), bf16_dev(k, d), bf16_dev(v, d), to_dev(g, d), to_dev(b, d), *meta, to_dev(state, d),
                        tree_mask=mask, scale=1.0, max_nodes=FORMS[form])
    torch.cuda.synchronize()
    assert tl.last_kernel_name() == KERNEL.get(form, "delta_scan")
    got = f64(out)
    tol = 8 * F32_HALF * 2.02 * cols + BF16_HALF * left * cols
    assert (np.abs(got[i2, 0] - want[i2, 0]) <= tol).all(), (got[i2, 0] / cols, left)


# A state that forgets slowly (0.997 a token: a chunk of 64 leaves 0.83 of it), against f32 sums.  A chunk rounds it 7 times
# (the decay, three parts of each of two products), root 2.6 for independent signs; over the chunks it remembers 1.8 times as
# much: 4.8 half steps.  An update u is off by K S (12 sums), R, T R (12) and its weight: root 5.1.  Together 7.0.
# tests/test_mixers_precision_cpu.py shows that a last part missing anywhere takes a state past this bound.
SLOW_TOL = 8 * F32_HALF


def slow_step(rng, T, Hk, G, Dk, Dv):
    """q, k, v, g, b and a state in f64, as the operator gets them."""
    unit = lambda y: y / np.sqrt((y * y).sum(-1, keepdims=True))
    q, k = (spec.bf16(unit(rng.standard_normal((T, Hk, Dk)) + 0.4)) for _ in "qk")
    v = spec.bf16(rng.standard_normal((T, Hk * G, Dv)))
    g = (-0.003 * np.exp(0.5 * rng.standard_normal((T, Hk * G)))).astype(np.float32)
    b = (1 / (1 + np.exp(-rng.standard_normal((T, Hk * G))))).astype(np.float32)
    return q, k, v, g, b, (0.3 * rng.standard_normal((1, Hk * G, Dk, Dv))).astype(np.float32)


@pytest.mark.parametrize("form,T,step", [("chunks", 2085, 2085), ("trees and chunks", 1100, 1100), ("chunks", 64, 64), ("one chunk", 640, 64),
                                         ("one chunk", 33, 33)])
@pytest.mark.parametrize("Hk,G,Dk,Dv", [(1, 2, 64, 48), (1, 2, 128, 48)])
def test_a_state_that_forgets_slowly(tl, torch, Hk, G, Dk, Dv, form, T, step):  # noqa: F811
    """Thousands of tokens through the chunks, in one call or in several: states within f32's roundings of the recurrence in
    64 bits; outputs within bfloat16's and, for what the sums leave (Q S 12 sums, the weights 4, the updates 7, P U 12), 35
    half steps of f32 of the magnitudes that were added."""
    announce(f"slow decays, {form}, {T} tokens by {step}, Dk={Dk}")
    d, rng = dev(), np.random.default_rng(T + Dk)
    q, k, v, g, b, state = slow_step(rng, T, Hk, G, Dk, Dv)
    stated = to_dev(state, d)
    outs = []
    for lo in range(0, T, step):
        at = slice(lo, lo + step)
        n = len(q[at])
        meta = [to_dev(np.array(x, np.int32), d) for x in ([0, n], [n + 9], [0])]
        mask = torch.zeros(n, dtype=torch.int64, device=d) if "trees" in form else None
        outs.append(tl.delta_rule(*(bf16_dev(x[at], d) for x in (q, k, v)), to_dev(g[at], d), to_dev(b[at], d), *meta, stated,
                                  tree_mask=mask, max_nodes=FORMS[form]))
        assert tl.last_kernel_name() == KERNEL.get(form, "delta_scan")
    torch.cuda.synchronize()
    want, after, size = ref.delta_rule(q, k, v, g.astype(np.float64), b.astype(np.float64), [0, T], [T + 9], [0],
                                       state.astype(np.float64), None, Dk ** -0.5, np.zeros((T, Hk * G, Dv)))
    for h in range(Hk * G):
        miss = np.linalg.norm(stated.cpu().numpy()[0, h] - after[0, h]) / np.linalg.norm(after[0, h])
        assert miss <= SLOW_TOL, (h, miss / F32_HALF)
    got = np.concatenate([f64(o) for o in outs])
    assert (np.abs(got - want) <= BF16_HALF * np.abs(want) + 35 * F32_HALF * size).all()
