"""The hybrid decoding example, in which all operators of a step run together, against its plain definition in 64 bits:
the logits of every token that it takes, whatever was drafted, and what it accepts of drafts that hold the answer."""
from __future__ import annotations

import importlib.util
import math
import os

import numpy as np
import pytest

from gpu_common import announce, dev
from oracle.hybrid import Decoder

pytestmark = pytest.mark.gpu

VOCAB, COUNT, DEPTH = 512, 20, 5
LENGTHS = (1, 17, 40)       # of the prompts: at most 64 tokens in a step, which the ternary layers take without rounding inputs to 8 bits
# How far the logits of the two (of size 1, root mean square over the vocabulary) may be apart.  Values are rounded to
# bfloat16 ten times a layer (two norms, the projection, what the mixer or the attention takes and gives, the norm of
# that, o, gate|up, their product, down) and once before the head: 31 times in three layers, by at most half of a step of
# 2^-7 to 2^-8 of the value, 2^-7 / sqrt 12 in the mean square at most.  The roundings are independent, and on both sides:
# sqrt(2 * 31) of that; twice it for gains above one.
TOL = 2 * math.sqrt(2 * 31) * 2.0 ** -7 / math.sqrt(12)
# An 8-bit cache rounds K and V, once each, to steps of 2^-3 on both sides, of values that may differ by a bfloat16 step:
# as if neither rounding were the same, in a branch that is half of the sum at most.
TOL_E4M3 = math.hypot(TOL, 0.5 * math.sqrt(2) * 2.0 ** -3 / math.sqrt(12))


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def both(example):
    """The example's decoder, and its plain definition for a bfloat16 and an 8-bit cache."""
    weights, real = [], example.tl.pack_weights

    def keep(codes, scales):
        weights.append((codes.cpu().numpy(), scales.cpu().numpy()))
        return real(codes, scales)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(example.tl, "pack_weights", keep)
        model = example.HybridDecoder(vocab=VOCAB, max_pos=256, device=dev())
    w = {name: getattr(model, name).cpu().numpy() for name in
         ("embed", "taps", "gates", "a_log", "dt_bias", "q_weight", "k_weight", "cos_sin")}
    fours = [weights[i:i + 4] for i in range(0, 12, 4)]
    shape = (example.HEADS, example.KV_HEADS, example.D, example.KEY_HEADS, example.VALUE_HEADS, example.DK, example.DV)
    assert len(weights) == 13
    return model, [Decoder(w, fours[:2], fours[2:], weights[12], shape, e4m3) for e4m3 in (False, True)]


@pytest.fixture(scope="module")
def prompts():
    rng = np.random.default_rng(15)
    return [rng.integers(0, VOCAB, n).tolist() for n in LENGTHS]


def apart(a, b):
    """Root mean square of the difference of rows of logits."""
    return np.sqrt(((a - b) ** 2).mean(-1))


@pytest.mark.parametrize("cache", ["bfloat16", "float8_e4m3fn"])
@pytest.mark.parametrize("drafts", ["none", "history", "answer"])
def test_logits_are_those_of_the_plain_decoder(example, both, prompts, monkeypatch, drafts, cache):
    import torch
    model, plain = both
    plain, tol = plain[cache != "bfloat16"], TOL if cache == "bfloat16" else TOL_E4M3
    seen, real = [], example.tl.tree_verify

    def answer(history, nodes):
        """What the plain decoder says next, between wrong branches at every depth."""
        tokens, parents = [history[-1]], [-1]
        for depth, token in enumerate(plain.greedy(history, DEPTH)):
            tokens += [(token + 1) % VOCAB, token]
            parents += [2 * depth, 2 * depth]
        return tokens, parents

    def keep(logits, tokens, parents, q_start):
        got = real(logits, tokens, parents, q_start)
        seen.append([x.cpu().numpy() for x in (logits, q_start, *got)])
        return got
    announce(f"hybrid_decode against the plain decoder, cache={cache} drafts={drafts}")
    more = {"none": dict(nodes=1), "history": dict(nodes=12), "answer": dict(nodes=2 * DEPTH + 1, draft=answer)}[drafts]
    monkeypatch.setattr(example.tl, "tree_verify", keep)
    said, steps = example.generate(model, prompts, COUNT, cache=getattr(torch, cache), **more)
    assert len(seen) == steps + 1 and all(len(s) == COUNT for s in said)

    want = [plain.rows(p + s, None)[0] for p, s in zip(prompts, said)]
    far, so_far, later = [], [[] for _ in prompts], []
    wrong_at = None
    for step, (logits, q_start, accepted, path, nxt, target) in enumerate(seen):
        for r, prompt in enumerate(prompts):
            for i in range(accepted[r]):
                row, at = q_start[r] + path[r, i], len(prompt) - 1 + len(so_far[r])
                if len(so_far[r]) < COUNT:
                    far.append(apart(logits[row].astype(np.float64), want[r][at]))
                    if r == 0 and wrong_at is not None:
                        later.append((at, logits[row].astype(np.float64)))
                    so_far[r].append(int(target[row]))
            if r == 0 and wrong_at is None and step:
                wrong_at = len(prompt) + len(so_far[0]) - 2          # the last token that this step committed
    assert so_far == said
    assert len(far) >= len(prompts) * COUNT and max(far) <= tol, max(far)
    if drafts == "none":
        assert len(seen) == COUNT
    if drafts == "answer":
        assert len(seen) <= COUNT // 2

    # the comparison can fail: were one token missing in the states after its step, later logits would differ
    lost = plain.rows(prompts[0] + said[0], None, {wrong_at})[0]
    differ = [apart(y, lost[at]) for at, y in later][:4]
    assert len(differ) == 4 and min(differ) > tol, differ
