"""The chunked delta rule in f32 on the CPU, its operands cut into bfloat16 parts as the kernels cut them: with all three
parts a state that forgets slowly stays within the bound that the GPU tests hold it to, and with any one operand's last
part missing it does not."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.mixers as ref
import oracle.speculative as spec
from test_gpu_mixers_precision import SLOW_TOL, slow_step

F = np.float32


def parts(x, count):
    """bfloat16 parts of f32 numbers: cut off, but for the second of two, which is rounded."""
    x, out = np.ascontiguousarray(x, F), []
    for i in range(count):
        cut = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(F) if count == 3 or i == 0 else spec.bf16(x).astype(F)
        out.append(cut)
        x = x - cut
    return out


def advance(k, v, g, b, S, of_state=3, of_solver=3, of_rest=3, of_updates=3):
    """The state [Dk, Dv] of one head after the chunks of its tokens; of_*: the parts of each f32 operand."""
    for t0 in range(0, len(k), 64):
        at = slice(t0, t0 + 64)
        K, V, D = k[at].astype(F), v[at].astype(F), np.cumsum(g[at].astype(np.float64))
        A = np.tril(b[at, None] * np.exp((D[:, None] - D).astype(F)) * (K @ K.T), -1).astype(F)
        T = np.eye(len(K), dtype=F)
        for i in range(1, len(K)):
            T[i] -= A[i, :i] @ T[:i]
        T = parts(T * b[at], of_solver)
        told = sum(K @ p for p in parts(S, of_state)[::-1])
        R = parts(V - np.exp(D).astype(F)[:, None] * told, of_rest)
        U = np.zeros_like(V)
        for i, j in ((2, 0), (1, 1), (0, 2), (1, 0), (0, 1), (0, 0)):
            if i < of_solver and j < of_rest:
                U += T[i] @ R[j]
        S = np.exp(D[-1]).astype(F) * S
        for p in parts(np.exp(D[-1] - D).astype(F)[:, None] * U, of_updates)[::-1]:
            S = S + K.T @ p
    return S


@pytest.mark.parametrize("missing", [None, "of_state", "of_solver", "of_rest", "of_updates"])
@pytest.mark.parametrize("T,Dk", [(2085, 64), (1100, 128), (64, 64), (64, 128), (33, 64)])
def test_the_bound_sees_a_missing_part(T, Dk, missing):
    q, k, v, g, b, state = slow_step(np.random.default_rng(T + Dk), T, 1, 2, Dk, 48)
    _, want, _ = ref.delta_rule(q, k, v, g.astype(np.float64), b.astype(np.float64), [0, T], [T + 9], [0],
                                state.astype(np.float64), None, 1.0, np.zeros((T, 2, 48)))
    for h in range(2):
        S = advance(k[:, 0], v[:, h], g[:, h], b[:, h], state[0, h], **({missing: 2} if missing else {}))
        miss = np.linalg.norm(S - want[0, h]) / np.linalg.norm(want[0, h])
        assert (miss > SLOW_TOL) == (missing is not None), miss * 2.0 ** 24
