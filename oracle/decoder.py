"""A small decoder of ternary layers in binary64, without a cache of pages, trees or kernels: each token
sees the ones before it.  It rounds to bfloat16 (and to 8-bit rows of K and V) where the program that
runs on the GPU stores such values, and nowhere else."""
from __future__ import annotations

import numpy as np

from oracle import ternary
from oracle.speculative import bf16, e4m3_code, e4m3_value, rotate


def _apply(w, x):
    return x @ w.T


class Decoder:
    """embed [vocab, hidden]; layers: four ternary weights (codes [N, K], scales [N, K / 128]) each, for
    q|k|v, the attention's output, gate|up and down; head: one weight; cos_sin [positions, D]."""

    def __init__(self, embed, layers, head, cos_sin, heads, kv_heads, D, e4m3=False):
        # W H x for the block rotation H, which is its own transpose: (H W^T)^T x
        dense = lambda w: ternary.rotate_exact(w[0].astype(np.float64) * np.repeat(w[1].astype(np.float64), 128, axis=1))
        self.embed, self.cos_sin = np.asarray(embed, dtype=np.float64), cos_sin
        self.layers, self.head = [[dense(w) for w in layer] for layer in layers], dense(head)
        self.heads, self.kv_heads, self.D, self.e4m3 = heads, kv_heads, D, e4m3

    @staticmethod
    def _norm(x):
        return bf16(x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6))

    def _stored(self, rows):
        """Rows of K or V as the cache holds them."""
        if not self.e4m3:
            return rows
        scale = (np.abs(rows).max(-1, keepdims=True).astype(np.float32) / np.float32(448))
        codes = e4m3_code(rows.astype(np.float32) / np.where(scale > 0, scale, 1))
        return e4m3_value(codes) * scale.astype(np.float64)

    def rows(self, tokens, state, instead=None):
        """Advances `state`, (K, V) [n, kv_heads, D] of each layer (None: nothing said yet), by tokens; returns the logits
        [len(tokens), vocab] and the new state.  instead: {position: (K, V) rows [kv_heads, D] of each layer} that
        later tokens see in the place of the right ones."""
        n0 = 0 if state is None else len(state[0][0])
        positions = np.arange(n0, n0 + len(tokens))
        x, out = self.embed[list(tokens)], []
        G, D, H = self.heads // self.kv_heads, self.D, self.kv_heads
        for layer, (qkv, o, gate_up, down) in enumerate(self.layers):
            y = bf16(_apply(qkv, self._norm(x))).reshape(len(tokens), -1, D)
            q = bf16(rotate(y[:, :self.heads], self.cos_sin, positions))
            k = self._stored(bf16(rotate(y[:, self.heads:self.heads + H], self.cos_sin, positions)))
            v = self._stored(y[:, self.heads + H:])
            if state is not None:
                k, v = np.concatenate([state[layer][0], k]), np.concatenate([state[layer][1], v])
            seen_k, seen_v = k.copy(), v.copy()
            for p, rows in (instead or {}).items():
                seen_k[p], seen_v[p] = rows[layer]
            a = np.zeros((len(tokens), self.heads, D))
            for i, p in enumerate(positions):
                kk, vv = seen_k[:p + 1].copy(), seen_v[:p + 1].copy()
                kk[p], vv[p] = k[p], v[p]                  # its own rows were right when it was new
                for h in range(H):
                    s = q[i, h * G:(h + 1) * G] @ kk[:, h].T * D ** -0.5
                    w = np.exp(s - s.max(-1, keepdims=True))
                    a[i, h * G:(h + 1) * G] = (w / w.sum(-1, keepdims=True)) @ vv[:, h]
            x = x + bf16(_apply(o, bf16(a).reshape(len(tokens), -1)))
            gate, up = np.split(bf16(_apply(gate_up, self._norm(x))), 2, axis=1)
            x = x + bf16(_apply(down, bf16(gate / (1 + np.exp(-gate)) * up)))
            out.append((k, v))
        return _apply(self.head, self._norm(x)), out

    def logits(self, tokens, at=None):
        """at: {position: token} whose rows stay where the right token's belong (a drafted token's that was not taken)."""
        y, state = self.rows(tokens, None)
        if not at:
            return y
        before = lambda p: [(k[:p], v[:p]) for k, v in state] if p else None
        rows = {p: [(k[p], v[p]) for k, v in self.rows([t], before(p))[1]] for p, t in at.items()}
        return self.rows(tokens, None, rows)[0]

    def greedy(self, history, count):
        """The `count` likeliest tokens after `history`, one after another."""
        y, state = self.rows(history, None)
        said = []
        for _ in range(count):
            said.append(int(np.argmax(y[-1])))
            y, state = self.rows(said[-1:], state)
        return said
