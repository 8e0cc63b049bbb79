"""The speculative-decoding example against its plain definition in 64 bits: the logits of every token that
it takes, whatever was drafted, and what it accepts of drafts that hold the answer."""
from __future__ import annotations

import numpy as np
import pytest

from decoder_common import TOL, TOL_E4M3, VOCAB, apart, load_example, models
from gpu_common import announce, dev

pytestmark = pytest.mark.gpu

COUNT, DEPTH = 25, 5
LENGTHS = (1, 16, 37)       # of the prompts: at most 64 tokens in a step, which the layers take without rounding inputs to 8 bits


@pytest.fixture(scope="module")
def example():
    return load_example()


@pytest.fixture(scope="module")
def both(example):
    with pytest.MonkeyPatch.context() as m:
        return models(example, m, dev())


@pytest.fixture(scope="module")
def prompts():
    rng = np.random.default_rng(5)
    return [rng.integers(0, VOCAB, n).tolist() for n in LENGTHS]


def run(example, model, prompts, monkeypatch, kind, **more):
    """generate() with every verification recorded: (tokens said, the verifications)."""
    seen, real = [], example.tl.tree_verify

    def keep(logits, tokens, parents, q_start):
        got = real(logits, tokens, parents, q_start)
        seen.append([x.cpu().numpy() for x in (logits, q_start, *got)])
        return got
    with monkeypatch.context() as m:
        m.setattr(example.tl, "tree_verify", keep)
        said, _, steps = example.generate(model, prompts, COUNT, cache=kind, **more)
    assert len(seen) == steps + 1 and all(len(s) == COUNT for s in said)
    return said, seen


def taken(prompts, said, seen):
    """[(request, step, position, its logits)] of every token taken, up to the last one said; the tokens that
    the verifications name are those said."""
    out, so_far = [], [[] for _ in prompts]
    for step, (logits, q_start, accepted, path, nxt, target) in enumerate(seen):
        np.testing.assert_array_equal(target, logits.argmax(1))
        for r, prompt in enumerate(prompts):
            base = len(prompt) - 1 + len(so_far[r])
            for i in range(accepted[r]):
                row = q_start[r] + path[r, i]
                if base + i < len(prompt) + COUNT:
                    out.append((r, step, base + i, logits[row].astype(np.float64)))
                so_far[r].append(int(target[row]))
            assert nxt[r] == so_far[r][-1]
            del so_far[r][COUNT:]
    assert so_far == said
    return out


@pytest.mark.parametrize("cache", ["bfloat16", "float8_e4m3fn"])
@pytest.mark.parametrize("drafts", ["none", "history", "answer"])
def test_logits_are_those_of_the_plain_decoder(example, both, prompts, monkeypatch, drafts, cache):
    import torch
    model, plain = both
    plain, tol, kind = plain[cache != "bfloat16"], TOL if cache == "bfloat16" else TOL_E4M3, getattr(torch, cache)
    rights = []

    def answer(history, nodes):
        """What the plain decoder says next, between wrong branches at every depth."""
        right = plain.greedy(history, DEPTH)
        rights.append(right)
        tokens, parents = [history[-1]], [-1]
        for depth, token in enumerate(right):
            tokens += [(token + 1) % VOCAB, token]
            parents += [2 * depth, 2 * depth]
        return tokens, parents
    announce(f"speculative_decode against the plain decoder, cache={cache} drafts={drafts}")
    more = {"none": dict(nodes=1), "history": dict(nodes=12), "answer": dict(nodes=2 * DEPTH + 1, draft=answer)}[drafts]
    said, seen = run(example, model, prompts, monkeypatch, kind, **more)
    rows = taken(prompts, said, seen)
    want = [plain.logits(p + s) for p, s in zip(prompts, said)]
    far = np.array([apart(y, want[r][at]) for r, _, at, y in rows])
    assert len(far) >= len(prompts) * COUNT and far.max() <= tol, far.max()

    if drafts == "none":
        assert len(seen) == COUNT
        return
    assert len(seen) <= COUNT
    if drafts == "history":
        return
    for step, (_, _, accepted, path, nxt, _) in enumerate(seen[1:]):
        for r in range(len(prompts)):
            right, n = rights[step * len(prompts) + r], int(accepted[r])
            np.testing.assert_array_equal(path[r, :n - 1], 2 * np.arange(n - 1))  # wrong branches have no children
            if path[r, n - 1] == 2 * (n - 1) and n <= DEPTH:                       # stopped: neither child was the answer
                assert nxt[r] not in (right[n - 1], (right[n - 1] + 1) % VOCAB)
    assert len(seen) <= COUNT // 2

    # the comparison can fail: with a wrong branch's row in the place of the first accepted one, later steps differ
    step, at = next((i, len(prompts[0]) - 1 + sum(int(s[2][0]) for s in seen[:i]) + 1)
                    for i in range(1, len(seen)) if seen[i][2][0] > 2)
    full = prompts[0] + said[0]
    wrong = plain.logits(full, {at: (full[at] + 1) % VOCAB})
    later = [apart(y, wrong[p]) for r, s, p, y in rows if r == 0 and s > step][:6]
    assert len(later) == 6 and min(later) > tol, later
