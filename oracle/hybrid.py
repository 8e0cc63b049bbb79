"""A small hybrid decoder of ternary layers in binary64: layers that keep a state (short convolution, gated delta
rule) and attention layers whose heads are normed before they are turned; token by token, without trees, pages,
chunks or kernels.  It rounds to bfloat16 (and to 8-bit rows of K and V) where the program that runs on the GPU
stores such values, and nowhere else."""
from __future__ import annotations

import numpy as np

from oracle import mixers, ternary
from oracle.speculative import bf16, e4m3_code, e4m3_value


def rms(x):
    return bf16(x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6))


class Decoder:
    """w: {"embed", "taps", "gates", "a_log", "dt_bias", "q_weight", "k_weight", "cos_sin"} as the program has them;
    mixers, attention: for each layer its four ternary weights (codes [N, K], scales [N, K / 128]); head: one;
    shape: (attention heads, their cache heads, D, key heads, value heads, Dk, Dv)."""

    def __init__(self, w, mixers_, attention, head, shape, e4m3=False):
        dense = lambda x: ternary.rotate_exact(x[0].astype(np.float64) * np.repeat(x[1].astype(np.float64), 128, axis=1)).T
        self.w = {name: np.asarray(x, dtype=np.float64) for name, x in w.items()}
        self.mixers, self.attention = ([[dense(x) for x in layer] for layer in layers] for layers in (mixers_, attention))
        self.head, self.shape, self.e4m3 = dense(head), shape, e4m3

    def _stored(self, rows, rounded):
        """Rows of K or V as the cache holds them."""
        if not self.e4m3:
            return bf16(rows) if rounded else rows
        scale = (np.abs(rows).max(-1, keepdims=True).astype(np.float32) / np.float32(448))
        codes = e4m3_code(rows.astype(np.float32) / np.where(scale > 0, scale, 1))
        return e4m3_value(codes) * scale.astype(np.float64)

    def _rest(self, x, mixed, o, gate_up, down):
        x = x + bf16(mixed @ o)
        gate, up = np.split(bf16(rms(x) @ gate_up), 2, axis=1)
        return x + bf16(bf16(gate / (1 + np.exp(-gate)) * up) @ down)

    def _mixer(self, x, layer, state, lost):
        *_, Hk, Hv, Dk, Dv = self.shape
        project, *rest = self.mixers[layer]
        w, h = self.w, rms(x)
        rows = bf16(h @ project)
        conv, S, n0 = state if state is not None else (np.zeros((w["taps"].shape[2] - 1, rows.shape[1])), np.zeros((Hv, Dk, Dv)), 0)
        a, b = np.split(h @ w["gates"][layer], 2, axis=1)
        g, b = mixers.gates(a, b, w["a_log"][layer], w["dt_bias"][layer])
        out = np.zeros((len(x), Hv, Dv))
        for i in range(len(x)):
            y = (np.concatenate([conv, rows[i:i + 1]]) * w["taps"][layer].T).sum(0)
            y = y / (1 + np.exp(-y))
            qk = y[:2 * Hk * Dk].reshape(2, Hk, Dk)
            q, k = bf16(qk / np.sqrt((qk * qk).sum(-1, keepdims=True) + 1e-6))
            q, k = (np.repeat(t, Hv // Hk, 0) for t in (q, k))
            v = bf16(y[2 * Hk * Dk:]).reshape(Hv, Dv)
            next_S = np.exp(g[i])[:, None, None] * S
            u = b[i][:, None] * (v - (next_S * k[:, :, None]).sum(1))
            next_S = next_S + k[:, :, None] * u[:, None, :]
            out[i] = Dk ** -0.5 * (next_S * q[:, :, None]).sum(1)
            if n0 + i not in lost:
                S, conv = next_S, np.concatenate([conv, rows[i:i + 1]])[1:]
        return self._rest(x, rms(bf16(out)).reshape(len(x), -1), *rest), (conv, S, n0 + len(x))

    def _attend(self, x, layer, state):
        heads, H, D, *_ = self.shape
        qkv, *rest = self.attention[layer]
        w, G = self.w, heads // H
        y = bf16(rms(x) @ qkv).reshape(len(x), -1, D)
        n0 = 0 if state is None else len(state[0])
        positions = np.arange(n0, n0 + len(x))[None]
        turned = lambda t, weight: mixers.turned(mixers.normed(t, weight[layer], 1e-6), w["cos_sin"], positions, None)
        q = bf16(turned(y[:, :heads], w["q_weight"]))
        k = self._stored(turned(y[:, heads:heads + H], w["k_weight"]), True)
        v = self._stored(y[:, heads + H:], False)
        if state is not None:
            k, v = np.concatenate([state[0], k]), np.concatenate([state[1], v])
        a = np.zeros((len(x), heads, D))
        for i, p in enumerate(positions[0]):
            for h in range(H):
                s = q[i, h * G:(h + 1) * G] @ k[:p + 1, h].T * D ** -0.5
                e = np.exp(s - s.max(-1, keepdims=True))
                a[i, h * G:(h + 1) * G] = (e / e.sum(-1, keepdims=True)) @ v[:p + 1, h]
        return self._rest(x, bf16(a).reshape(len(x), -1), *rest), (k, v)

    def rows(self, tokens, state, lost=()):
        """Logits [len(tokens), vocab] after `state` (None: nothing said yet), and the new state.  lost: positions
        whose tokens the states of the first kind of layer forget."""
        x, out = self.w["embed"][list(tokens)], []
        state = state or [None] * (len(self.mixers) + len(self.attention))
        for i in range(len(self.attention)):
            for layer in (2 * i, 2 * i + 1):
                x, s = self._mixer(x, layer, state[len(out)], lost)
                out.append(s)
            x, s = self._attend(x, i, state[len(out)])
            out.append(s)
        return rms(x) @ self.head, out

    def greedy(self, history, count):
        """The `count` likeliest tokens after `history`, one after another."""
        y, state = self.rows(history, None)
        said = []
        for _ in range(count):
            said.append(int(np.argmax(y[-1])))
            y, state = self.rows(said[-1:], state)
        return said
