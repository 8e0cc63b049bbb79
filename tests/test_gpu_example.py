"""The speculative-decoding example: the library's calls run together as a program uses them."""
from __future__ import annotations

import importlib.util
import os

import pytest

from gpu_common import announce

pytestmark = pytest.mark.gpu

COUNT, DEPTH = 25, 5


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def model(example):
    return example.Decoder(layers=2, vocab=512, max_pos=256)


def _same_until_a_tie(want, lead, got):
    """Both runs round the same sums in other orders: a bfloat16 may come out a step (2^-7) apart.  About ten
    values a layer are rounded on the way, two layers, and the last norm: the logits, of size 1, are off by
    21 2^-7 at the very most, and two of them change places only where they are closer than twice that."""
    for a, margin, b in zip(want, lead, got):
        for x, m, y in zip(a, margin, b):
            if x != y:
                assert m <= 2 * 21 * 2.0 ** -7
                break


@pytest.mark.parametrize("cache", ["bfloat16", "float8_e4m3fn"])
def test_trees_decode_what_single_tokens_decode(example, model, cache):
    import torch
    kind = getattr(torch, cache)
    gen = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, 512, (n,), generator=gen).tolist() for n in (1, 16, 37, 120)]
    announce(f"speculative_decode cache={cache} one token a step")
    want, lead, steps = example.generate(model, prompts, COUNT, 1, kind)
    assert steps == COUNT - 1 and all(len(s) == COUNT for s in want)

    announce(f"speculative_decode cache={cache} drafts from the history")
    got, _, steps = example.generate(model, prompts, COUNT, 12, kind)
    assert steps <= COUNT - 1 and all(len(s) == COUNT for s in got)
    _same_until_a_tie(want, lead, got)

    def known(history, nodes):
        """The right continuation between wrong branches at every depth."""
        r = next(i for i, p in enumerate(prompts) if history[:len(p)] == p)
        said = len(history) - len(prompts[r])
        right = want[r][said:said + DEPTH]
        tokens, parents, at = [history[-1]], [-1], 0
        for token in right:
            tokens += [(token + 1) % 512, token]
            parents += [at, at]
            at = len(tokens) - 1
        return tokens, parents

    announce(f"speculative_decode cache={cache} drafts that hold the answer")
    got, _, steps = example.generate(model, prompts, COUNT, 2 * DEPTH + 1, kind, draft=known)
    _same_until_a_tie(want, lead, got)
    if got == want:
        assert steps == -(-(COUNT - 1) // (DEPTH + 1))
