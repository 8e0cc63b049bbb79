"""Greedy decoding of several requests with drafted trees, over one paged K/V cache: a small
decoder of ternary linear layers with random weights, on one MI355X.

    python examples/speculative_decode.py --requests 4 --tokens 64 --cache e4m3

Each step drafts, for every request, a tree of guesses from what the request has said before,
runs all trees through the model at once and keeps the longest branch that greedy decoding
would have taken.  The library's part of a step, in order:

    step_plan       pages for the step's tokens, their slots, positions and tree masks
    per layer:      linear_apply (qkv), kv_write (rotary embedding, cache), tree_attention,
                    linear_apply (o, gate_up, down)
    tree_verify     the accepted branch of each tree and the token after it
    kv_commit       the accepted rows to their places after the context, in every layer

The host reads back the accepted branches once a step, because the drafts are made there.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_gemv_gemm_amd as tl  # noqa: E402

HIDDEN, MLP, HEADS, KV_HEADS, D = 1024, 2048, 8, 2, 128


class Linear:
    """A ternary layer with random codes, scaled to keep its input's size."""

    def __init__(self, K, N, gen, device):
        codes = torch.randint(-1, 2, (N, K), dtype=torch.int8, generator=gen).to(device)
        scales = (torch.rand((N, K // 128), generator=gen) * 0.5 + 0.75) * (1.5 / K) ** 0.5
        self.scales = scales.to(torch.float16).to(device)
        self.packed, self.q, self.row_scale = tl.pack_weights(codes, self.scales)

    def __call__(self, x, dtype=torch.bfloat16):
        return tl.linear_apply(x, self.packed, self.scales, self.q, self.row_scale, out_dtype=dtype)


class Decoder:
    def __init__(self, layers=2, vocab=512, max_pos=4096, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        self.device, self.layers, self.vocab = device, layers, vocab
        self.embed = torch.randn((vocab, HIDDEN), generator=gen).to(device)
        sizes = ((HIDDEN, (HEADS + 2 * KV_HEADS) * D), (HEADS * D, HIDDEN), (HIDDEN, 2 * MLP), (MLP, HIDDEN))
        self.blocks = [[Linear(K, N, gen, device) for K, N in sizes] for _ in range(layers)]
        self.head = Linear(HIDDEN, vocab, gen, device)
        angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(D // 2, dtype=torch.float64) / (D // 2))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)

    @staticmethod
    def _norm(x):
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def forward(self, tokens, plan, state, max_nodes):
        """Logits f32 [T, vocab] of the step's tokens; their keys and values go to the cache."""
        q_start, kv_lens, slots, positions, mask = plan
        x = self.embed[tokens.long()]
        for layer, (qkv, o, gate_up, down) in enumerate(self.blocks):
            k_cache, v_cache, k_scale, v_scale = (None if c is None else c[layer] for c in state.cache)
            q, k, v = qkv(self._norm(x)).unflatten(1, (HEADS + 2 * KV_HEADS, D)).split((HEADS, KV_HEADS, KV_HEADS), 1)
            q = tl.kv_write(k, v, slots, k_cache, v_cache, k_scale, v_scale, q=q, positions=positions,
                            cos_sin=self.cos_sin)
            a = tl.tree_attention(q, k_cache, v_cache, state.table, q_start, kv_lens, tree_mask=mask, k_scale=k_scale,
                                  v_scale=v_scale, max_nodes=max_nodes)
            x = x + o(a.flatten(1)).float()
            gate, up = gate_up(self._norm(x)).float().chunk(2, 1)
            x = x + down((gate * torch.sigmoid(gate) * up).to(torch.bfloat16)).float()
        return self.head(self._norm(x), torch.float32)


class State:
    """The requests' pages: a table of them, how many each has, and the list of free ones."""

    def __init__(self, model, requests, capacity, block=16, dtype=torch.bfloat16):
        d, width = model.device, -(-capacity // block)
        pages = requests * width
        self.block, self.ints = block, dict(dtype=torch.int32, device=d)
        self.cache = tl.kv_cache(pages, KV_HEADS, block, D, dtype, layers=model.layers, device=d)
        self.table = torch.full((requests, width), -1, **self.ints)
        self.owned = torch.zeros(requests, **self.ints)
        self.ctx = torch.zeros(requests, **self.ints)
        self.free, self.head = torch.randperm(pages).to(**self.ints), torch.zeros(1, **self.ints)

    def plan(self, new, parents=None):
        new_lens = torch.tensor(new, **self.ints)
        *plan, self.owned, self.head = tl.step_plan(self.ctx, new_lens, self.owned, self.table, self.free, self.head,
                                                    sum(new), self.block, parents)
        return plan


def draft_tree(history, nodes, depth=6, branches=4):
    """Tokens and parents (-1: the root) of a tree below the last token of `history`: what followed
    it at its latest earlier places, the places where two tokens match first."""
    tokens, parents, child = [history[-1]], [-1], {}
    places = [i for i in range(len(history) - 2, -1, -1) if history[i] == history[-1]]
    places.sort(key=lambda i: not (i > 0 and len(history) > 1 and history[i - 1] == history[-2]))
    for i in places[:branches]:
        at = 0
        for token in history[i + 1:i + 1 + depth]:
            if (at, token) not in child:
                if len(tokens) == nodes:
                    break
                child[at, token] = len(tokens)
                tokens.append(token)
                parents.append(at)
            at = child[at, token]
    return tokens, parents


@torch.no_grad()
def generate(model, prompts, count, nodes=16, cache=torch.bfloat16, draft=draft_tree):
    """`count` tokens after each prompt, with trees of up to `nodes` tokens (1: one token a step).
    Returns the tokens, for each its logit's lead over the next best, and the steps taken."""
    R, capacity = len(prompts), max(map(len, prompts)) + count + 2 * nodes
    if capacity > len(model.cos_sin):                    # kv_write clamps positions to the table
        raise ValueError(f"{capacity} positions are needed, the model's rotary table has {len(model.cos_sin)}")
    state = State(model, R, capacity, dtype=cache)
    ints = state.ints

    def verify(logits, tokens, parents, q_start):
        accepted, path, nxt, target = tl.tree_verify(logits, tokens, parents, q_start)
        top = logits.topk(2).values
        return accepted, path, nxt, torch.cat([accepted, nxt]).tolist(), path.tolist(), (top[:, 0] - top[:, 1]).tolist()

    # the prompts, as chains; one row of logits for each
    lens = [len(p) for p in prompts]
    plan = state.plan(lens)
    tokens = torch.tensor([t for p in prompts for t in p], **ints)
    logits = model.forward(tokens, plan, state, max(lens))
    last = (plan[0][1:] - 1).long()
    *_, found, _, lead = verify(logits[last], tokens[last], torch.full((R,), -1, **ints), torch.arange(R + 1, **ints))
    state.ctx = plan[1]
    said = [[t] for t in found[R:]]
    leads, steps = [[x] for x in lead], 0

    while min(map(len, said)) < count:
        trees = [draft(prompts[r] + said[r], nodes) for r in range(R)]
        sizes = [len(t) for t, _ in trees]
        tokens = torch.tensor([t for tree, _ in trees for t in tree], **ints)
        parents = torch.tensor([p for _, tree in trees for p in tree], **ints)
        plan = state.plan(sizes, parents)
        logits = model.forward(tokens, plan, state, max(sizes))
        accepted, path, nxt, found, paths, lead = verify(logits, tokens, parents, plan[0])
        state.ctx = tl.kv_commit(accepted, path, state.ctx, plan[1], state.table, *state.cache)
        first = 0
        for r, (tree, _) in enumerate(trees):
            taken = paths[r][:found[r]]
            said[r] += [tree[i] for i in taken[1:]] + [found[R + r]]
            leads[r] += [lead[first + i] for i in taken]
            first += sizes[r]
            cut = len(said[r]) - count
            if cut > 0:                                  # a request that is done waits for the others
                del said[r][count:], leads[r][count:]
                state.ctx[r] -= cut
        steps += 1
    return said, leads, steps


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
    model = Decoder()
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (max(1, args.prompt - 3 * r),), generator=gen).tolist()
               for r in range(args.requests)]
    cache = torch.float8_e4m3fn if args.cache == "e4m3" else torch.bfloat16
    for nodes in (1, args.nodes):
        generate(model, prompts, 4, nodes, cache)        # the first launches
        torch.cuda.synchronize()
        start = time.perf_counter()
        _, _, steps = generate(model, prompts, args.tokens, nodes, cache)
        torch.cuda.synchronize()
        took = time.perf_counter() - start
        print(f"trees of up to {nodes:2d} tokens: {args.requests} x {args.tokens} tokens in {steps} steps, "
              f"{(args.tokens - 1) / max(steps, 1):.2f} tokens a step, {1e3 * took / max(steps, 1):.2f} ms a step")


if __name__ == "__main__":
    main()
