"""How exact the gated delta rule's outputs and states are: outputs whose large terms cancel, so that what is left would be
gone if an operand had lost its last bits, in every form of the operator."""
from __future__ import annotations

import numpy as np
import pytest

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
