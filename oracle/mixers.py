"""Plain definitions of the normed cache write, the short convolution, the gated delta rule and the commit of its
states, token by token in numpy (binary64), written from the formulas alone."""
from __future__ import annotations

import numpy as np

NODES = 64


def normed(x, weight, eps):
    """Rows x [.., D] times weight [D] (None: ones) over the root of their mean square."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if weight is None else y * weight


def turned(x, cos_sin, positions, axis_of):
    """Rows x [T, heads, D] turned in pairs (d, d + rot / 2) by positions [axes, T] of the pair's axis."""
    h = cos_sin.shape[1] // 2
    most = cos_sin.shape[0] - 1
    y = x.copy()
    for d in range(h):
        axis = 0 if axis_of is None else min(max(int(axis_of[d]), 0), len(positions) - 1)
        at = np.clip(positions[axis], 0, most)
        c, s = (cos_sin[at, j].astype(np.float64)[:, None] for j in (d, d + h))
        y[..., d], y[..., d + h] = x[..., d] * c - x[..., d + h] * s, x[..., d + h] * c + x[..., d] * s
    return y


def good_starts(q_start, T):
    return q_start[0] >= 0 and q_start[-1] <= T and all(a <= b for a, b in zip(q_start, q_start[1:]))


def requests(q_start, kv_lens, slots, states, T):
    """(first, n, row of the state or -1, whether it has just begun) of each request with tokens."""
    if not good_starts(q_start, T):
        return
    for r, kv in enumerate(kv_lens):
        first, n = int(q_start[r]), int(q_start[r + 1] - q_start[r])
        if n > 0:
            row = int(slots[r]) if kv > 0 and 0 <= slots[r] < states else -1
            yield r, first, n, row, kv <= n


def ancestors(word, i):
    """Numbers of a tree node's ancestors and its own, rising."""
    word = int(word) & ((2 << i) - 1) | 1 << i
    return [j for j in range(i + 1) if word >> j & 1]


def lines(n, tree, mask):
    """For each token its ancestors and itself: all tokens up to it, or what the mask says."""
    return [ancestors(mask[i], i) if tree else list(range(i + 1)) for i in range(n)]


def short_conv(x, weight, bias, q_start, kv_lens, slots, state, mask, heads, dim, eps, out):
    """Returns out [T, C] (given: what was there before), the state after, and for every output the error that f32
    sums leave, in half steps of f32."""
    T, C = x.shape
    taps = weight.shape[1]
    out, after, err = out.copy(), state.copy(), np.zeros(out.shape)
    for r, first, n, row, fresh in requests(q_start, kv_lens, slots, len(state), T):
        if row < 0:
            out[first:first + n] = 0
            continue
        old = np.zeros_like(state[row]) if fresh else state[row]
        tree = mask is not None and n <= NODES
        for i in range(n):
            line = ancestors(mask[first + i], i) if tree else [i - j for j in range(taps - 1, -1, -1) if i >= j]
            line = line[-taps:]
            rows = [x[first + j] for j in line]
            rows = list(old[len(old) - (taps - len(rows)):] if taps > len(rows) else []) + rows
            y = sum(weight[:, j] * rows[j] for j in range(taps)) + (0 if bias is None else bias)
            size = sum(np.abs(weight[:, j] * rows[j]) for j in range(taps)) + (0 if bias is None else np.abs(bias))
            # each of the sum's terms is rounded once; y / (1 + exp(-y)) has a slope of at most 1.1; exp's argument is off
            # by two half steps, exp itself, the reciprocal (a step each), the sum and the product by six more
            z = y / (1 + np.exp(-y))
            e = 1.1 * (taps + 1) * size + (6 + 2 * np.abs(y)) * np.abs(z)
            for h in range(heads):
                c = slice(h * dim, (h + 1) * dim)
                length = np.sqrt((z[c] ** 2).sum() + eps)
                # the length is off by what its parts are (at most the root of their squares' sum), by the sum's own
                # roundings (dim / 8 + 8 of them) and the root, the division and the product
                e[c] = e[c] / length + np.abs(z[c]) / length * (np.sqrt((e[c] ** 2).sum()) / length + dim / 8 + 8 + 4)
                z[c] = z[c] / length
            out[first + i], err[first + i] = z, e
        if not tree:
            after[row] = np.concatenate([old, x[first:first + n]])[-(taps - 1):]
    return out, after, err


def gates(a, b, a_log, dt_bias):
    """Log decay and step from a layer's columns."""
    z = a + dt_bias
    return -np.exp(a_log) * (np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z)))), 1 / (1 + np.exp(-b))


def delta_rule(q, k, v, g, b, q_start, kv_lens, slots, state, mask, scale, out):
    """Returns out [T, Hv, Dv] (given: what was there before), the states after, and the sum of magnitudes of the terms
    of every output, all in 64 bits.  u_i = b_i (v_i - exp(D_i) S^T k_i - sum over ancestors j of
    exp(D_i - D_j) (k_i k_j) u_j) with D the sum of g over the token and its ancestors."""
    T, Hv, Dv = v.shape
    G = Hv // q.shape[1]
    out, after, size = out.copy(), state.copy(), np.zeros(out.shape)
    k, q = np.repeat(k, G, 1), np.repeat(q, G, 1)
    g = np.maximum(g, -1e4)
    for r, first, n, row, fresh in requests(q_start, kv_lens, slots, len(state), T):
        if row < 0:
            out[first:first + n] = 0
            continue
        S = np.zeros_like(state[row]) if fresh else state[row]
        if mask is not None and n <= NODES:
            u, D = np.zeros((n, Hv, Dv)), np.zeros((n, Hv))
            for i in range(n):
                t, line = first + i, ancestors(mask[first + i], i)
                D[i] = sum(g[first + j] for j in line)
                told = np.einsum("hkd,hk->hd", S, k[t])
                u[i] = v[t] - np.exp(D[i])[:, None] * told
                for j in line[:-1]:
                    u[i] -= (np.exp(D[i] - D[j]) * (k[t] * k[first + j]).sum(-1))[:, None] * u[j]
                u[i] *= b[t][:, None]
                o = np.exp(D[i])[:, None] * np.einsum("hkd,hk->hd", S, q[t])
                big = np.exp(D[i])[:, None] * np.einsum("hkd,hk->hd", np.abs(S), np.abs(q[t]))
                for j in line:
                    w = (np.exp(D[i] - D[j]) * (q[t] * k[first + j]).sum(-1))[:, None]
                    o += w * u[j]
                    big += (np.exp(D[i] - D[j]) * np.abs(q[t] * k[first + j]).sum(-1))[:, None] * np.abs(u[j])
                out[t], size[t] = scale * o, abs(scale) * big
            continue
        A = np.abs(S)
        for t in range(first, first + n):
            e = np.exp(g[t])[:, None, None]
            S = e * S
            u = b[t][:, None] * (v[t] - np.einsum("hkd,hk->hd", S, k[t]))
            S = S + k[t][:, :, None] * u[:, None, :]
            A = e * A + np.abs(k[t])[:, :, None] * np.abs(u)[:, None, :]
            out[t] = scale * np.einsum("hkd,hk->hd", S, q[t])
            size[t] = abs(scale) * np.einsum("hkd,hk->hd", A, np.abs(q[t]))
        after[row] = S
    return out, after, size


def delta_commit(accepted, path, q_start, kv_lens, slots, k, v, g, b, state, x, conv_state):
    """The states [states, ..] of one layer after the accepted branches: the chain of the branch's tokens."""
    after, conv = state.copy(), conv_state.copy()
    for r, first, n, row, fresh in requests(q_start, kv_lens, slots, len(state), len(k)):
        nodes = [int(p) for p in path[r][:max(int(accepted[r]), 0)] if 0 <= p < n] if n <= NODES and row >= 0 else []
        if not nodes:
            continue
        at = [first + p for p in nodes]
        zero = np.zeros((len(at),) + v.shape[1:])
        start = np.zeros_like(state[row:row + 1]) if fresh else state[row:row + 1]
        _, S, _ = delta_rule(k[at], k[at], v[at], g[at], b[at], [0, len(at)], [len(at) + 1], [0], start, None, 1.0, zero)
        after[row] = S[0]
        old = np.zeros_like(conv_state[row]) if fresh else conv_state[row]
        conv[row] = np.concatenate([old, x[at]])[-len(old):]
    return after, conv
