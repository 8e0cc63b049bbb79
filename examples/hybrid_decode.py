"""Greedy decoding with drafted trees for a hybrid decoder: two layers that keep a state per request (short
convolution and gated delta rule) for each attention layer, all of ternary linear layers with random weights,
on one MI355X.

    python examples/hybrid_decode.py --requests 4 --tokens 64 --cache e4m3

The library's part of a step, in order:

    step_plan            pages for the step's tokens, their slots, positions and tree masks
    per state layer:     linear_apply (q|k|v), short_conv, delta_rule, linear_apply (o, gate_up, down)
    per attention layer: linear_apply (qkv), kv_write_norm (norms, rotary embedding, cache), tree_attention,
                         linear_apply (o, gate_up, down)
    tree_verify          the accepted branch of each tree and the token after it
    kv_commit            the accepted rows to their places after the context, in every attention layer
    delta_commit         the states along the accepted branches, in every state layer

A prompt is a chain: its states are there when the step is done.  A tree leaves the states alone, since no one
knows yet which branch is taken, and they move with delta_commit.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from speculative_decode import D, HEADS, HIDDEN, KV_HEADS, MLP, Linear, State, draft_tree  # noqa: E402

import quantized_gemv_gemm_amd as tl  # noqa: E402

KEY_HEADS, GROUP, DK, DV, TAPS = 2, 4, 128, 128, 4
VALUE_HEADS = KEY_HEADS * GROUP
QK, CHANNELS = KEY_HEADS * DK, 2 * KEY_HEADS * DK + VALUE_HEADS * DV


class HybridDecoder:
    def __init__(self, blocks=1, vocab=512, max_pos=4096, seed=0, device="cuda"):
        """`blocks` times two state layers and one attention layer."""
        gen = torch.Generator().manual_seed(seed)
        self.device, self.layers, self.state_layers, self.vocab = device, blocks, 2 * blocks, vocab
        normal = lambda *shape: torch.randn(shape, generator=gen).to(device)
        self.embed = normal(vocab, HIDDEN)
        mlp = ((HIDDEN, 2 * MLP), (MLP, HIDDEN))
        linears = lambda *sizes: [Linear(K, N, gen, device) for K, N in sizes]
        self.mixers = [linears((HIDDEN, CHANNELS), (VALUE_HEADS * DV, HIDDEN), *mlp) for _ in range(2 * blocks)]
        self.attention = [linears((HIDDEN, (HEADS + 2 * KV_HEADS) * D), (HEADS * D, HIDDEN), *mlp) for _ in range(blocks)]
        self.head = Linear(HIDDEN, vocab, gen, device)
        L = self.state_layers
        self.taps = normal(L, CHANNELS, TAPS) * TAPS ** -0.5
        self.gates = normal(L, HIDDEN, 2 * VALUE_HEADS) * HIDDEN ** -0.5     # a and b of every head
        self.a_log, self.dt_bias = normal(L, VALUE_HEADS) - 2, normal(L, VALUE_HEADS)
        self.q_weight, self.k_weight = 1 + 0.1 * normal(blocks, D), 1 + 0.1 * normal(blocks, D)
        angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(D // 4, dtype=torch.float64) / (D // 4))           # half of a head is turned
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)

    @staticmethod
    def _norm(x):
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def _mixer(self, x, layer, plan, state, max_nodes):
        q_start, kv_lens, _, _, mask = plan
        project, o, gate_up, down = self.mixers[layer]
        h = self._norm(x)
        into, y, ab = (t[layer] for t in state.step)
        into.copy_(project(h))
        torch.matmul(h.float(), self.gates[layer], out=ab)
        tl.short_conv(into, self.taps[layer], q_start, kv_lens, state.slots, state.conv[layer], tree_mask=mask,
                      norm_heads=2 * KEY_HEADS, norm_dim=DK, out=y)
        q, k, v = parts(y)
        u = tl.delta_rule(q, k, v, *ab.chunk(2, 1), q_start, kv_lens, state.slots, state.delta[layer], self.a_log[layer],
                          self.dt_bias[layer], tree_mask=mask, max_nodes=max_nodes)
        return self._rest(x, self._norm(u.float()).flatten(1), o, gate_up, down)

    def _attend(self, x, layer, plan, state, max_nodes):
        q_start, kv_lens, slots, positions, mask = plan
        qkv, o, gate_up, down = self.attention[layer]
        k_cache, v_cache, k_scale, v_scale = (None if c is None else c[layer] for c in state.cache)
        q, k, v = qkv(self._norm(x)).unflatten(1, (HEADS + 2 * KV_HEADS, D)).split((HEADS, KV_HEADS, KV_HEADS), 1)
        q = tl.kv_write_norm(k, v, slots, k_cache, v_cache, k_scale, v_scale, q=q, q_weight=self.q_weight[layer],
                             k_weight=self.k_weight[layer], positions=positions, cos_sin=self.cos_sin)
        a = tl.tree_attention(q, k_cache, v_cache, state.table, q_start, kv_lens, tree_mask=mask, k_scale=k_scale,
                              v_scale=v_scale, max_nodes=max_nodes)
        return self._rest(x, a.flatten(1), o, gate_up, down)

    def _rest(self, x, mixed, o, gate_up, down):
        x = x + o(mixed).float()
        gate, up = gate_up(self._norm(x)).float().chunk(2, 1)
        return x + down((gate * torch.sigmoid(gate) * up).to(torch.bfloat16)).float()

    def forward(self, tokens, plan, state, max_nodes):
        """Logits f32 [T, vocab]; keys and values go to the cache, a chain's states forward, and what a tree's
        commit needs of the state layers to state.step."""
        L, T = self.state_layers, len(tokens)
        kinds = ((CHANNELS, torch.bfloat16), (CHANNELS, torch.bfloat16), (2 * VALUE_HEADS, torch.float32))
        state.step = [torch.empty((L, T, n), dtype=t, device=self.device) for n, t in kinds]
        x = self.embed[tokens.long()]
        for layer in range(self.layers):
            x = self._mixer(x, 2 * layer, plan, state, max_nodes)
            x = self._mixer(x, 2 * layer + 1, plan, state, max_nodes)
            x = self._attend(x, layer, plan, state, max_nodes)
        return self.head(self._norm(x), torch.float32)

    def commit(self, accepted, path, plan, state):
        """The accepted branches' rows and states to where the next step looks for them."""
        q_start, kv_lens, *_ = plan
        into, y, ab = state.step
        _, k, v = parts(y)
        tl.delta_commit(accepted, path, q_start, kv_lens, state.slots, k, v, *ab.chunk(2, 2), state.delta, self.a_log,
                        self.dt_bias, x=into, conv_state=state.conv)
        state.ctx = tl.kv_commit(accepted, path, state.ctx, kv_lens, state.table, *state.cache)


def parts(y):
    """q, k and v [.., tokens, heads, width] of the convolution's channels."""
    return [t.unflatten(-1, (-1, n)) for t, n in zip(y.split((QK, QK, VALUE_HEADS * DV), -1), (DK, DK, DV))]


class HybridState(State):
    """Pages for the attention layers, and a row of states for each request."""

    def __init__(self, model, requests, capacity, **more):
        super().__init__(model, requests, capacity, **more)
        L, d = model.state_layers, model.device
        self.slots = torch.randperm(requests).to(**self.ints)
        # what a row holds before its request begins does not matter
        self.conv = torch.full((L, requests, TAPS - 1, CHANNELS), float("nan"), dtype=torch.bfloat16, device=d)
        self.delta = torch.full((L, requests, VALUE_HEADS, DK, DV), float("nan"), device=d)


@torch.no_grad()
def generate(model, prompts, count, nodes=16, cache=torch.bfloat16, draft=draft_tree):
    """`count` tokens after each prompt, with trees of up to `nodes` tokens (1: one token a step).
    Returns the tokens and the steps taken."""
    R, capacity = len(prompts), max(map(len, prompts)) + count + 2 * nodes
    if capacity > len(model.cos_sin):                    # kv_write_norm clamps positions to the table
        raise ValueError(f"{capacity} positions are needed, the model's rotary table has {len(model.cos_sin)}")
    state = HybridState(model, R, capacity, dtype=cache)
    ints = state.ints

    # the prompts, as chains; one row of logits for each
    lens = [len(p) for p in prompts]
    plan = state.plan(lens)
    tokens = torch.tensor([t for p in prompts for t in p], **ints)
    logits = model.forward(tokens, plan, state, max(lens))
    last = (plan[0][1:] - 1).long()
    _, _, nxt, _ = tl.tree_verify(logits[last], tokens[last], torch.full((R,), -1, **ints), torch.arange(R + 1, **ints))
    state.ctx = plan[1]
    said, steps = [[t] for t in nxt.tolist()], 0

    while min(map(len, said)) < count:
        # a request that is done has no tokens in the step
        trees = [draft(p + s, nodes) if len(s) < count else ([], []) for p, s in zip(prompts, said)]
        sizes = [len(t) for t, _ in trees]
        tokens = torch.tensor([t for tree, _ in trees for t in tree], **ints)
        parents = torch.tensor([p for _, tree in trees for p in tree], **ints)
        plan = state.plan(sizes, parents)
        logits = model.forward(tokens, plan, state, max(sizes))
        accepted, path, nxt, _ = tl.tree_verify(logits, tokens, parents, plan[0])
        model.commit(accepted, path, plan, state)
        found, paths = torch.cat([accepted, nxt]).tolist(), path.tolist()
        for r, (tree, _) in enumerate(trees):
            if tree:
                said[r] = (said[r] + [tree[i] for i in paths[r][1:found[r]]] + [found[R + r]])[:count]
        steps += 1
    return said, steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=48)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--nodes", type=int, default=16)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    args = ap.parse_args()
    if not 1 <= args.nodes <= tl.TREE_NODES:
        ap.error(f"--nodes must be 1 to {tl.TREE_NODES}")
    model = HybridDecoder()
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (max(1, args.prompt - 3 * r),), generator=gen).tolist()
               for r in range(args.requests)]
    cache = torch.float8_e4m3fn if args.cache == "e4m3" else torch.bfloat16
    for nodes in (1, args.nodes):
        generate(model, prompts, 4, nodes, cache)        # the first launches
        torch.cuda.synchronize()
        start = time.perf_counter()
        _, steps = generate(model, prompts, args.tokens, nodes, cache)
        torch.cuda.synchronize()
        took = time.perf_counter() - start
        print(f"trees of up to {nodes:2d} tokens: {args.requests} x {args.tokens} tokens in {steps} steps, "
              f"{(args.tokens - 1) / max(steps, 1):.2f} tokens a step, {1e3 * took / max(steps, 1):.2f} ms a step")


if __name__ == "__main__":
    main()
