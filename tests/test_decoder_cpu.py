"""The plain decoder that the example is compared with: its steps, and whether the comparison can fail."""
from __future__ import annotations

import numpy as np
import pytest

pytest.importorskip("torch")
from decoder_common import MAX_POS, TOL, TOL_E4M3, VOCAB, apart, load_example, models  # noqa: E402


@pytest.fixture(scope="module")
def example():
    return load_example()


@pytest.fixture(scope="module")
def both(example):
    with pytest.MonkeyPatch.context() as m:
        return models(example, m, "cpu", pack=lambda codes, scales: (None, None, None))


@pytest.fixture(scope="module")
def plain(both):
    return both[1]


def test_the_example_refuses_what_its_rotary_table_lacks(example, both):
    """Positions past the table would all be turned as its last one is."""
    prompts = [[1, 2, 3], [4] * 200]
    with pytest.raises(ValueError, match="positions"):
        example.generate(both[0], prompts, MAX_POS - 200 - 16 + 1, nodes=8)
    with pytest.raises(ValueError, match="positions"):
        example.generate(both[0], [[0] * MAX_POS], 1, nodes=1)


def test_tokens_one_at_a_time_are_tokens_at_once(plain):
    tokens = np.random.default_rng(0).integers(0, VOCAB, 18).tolist()
    for p in plain:
        whole = p.logits(tokens)
        first, state = p.rows(tokens[:7], None)
        second, state = p.rows(tokens[7:8], state)
        third, _ = p.rows(tokens[8:], state)
        assert np.abs(np.concatenate([first, second, third]) - whole).max() < 1e-9
        assert p.greedy(tokens[:7], 1) == [int(np.argmax(whole[6]))]


@pytest.mark.parametrize("which,tol", [(0, TOL), (1, TOL_E4M3)])
def test_rows_of_another_token_show(plain, which, tol):
    """One row of K and V that belongs to a token that was not taken, at several places: every token of the
    next few differs by more than twice the tolerance, none before."""
    rng = np.random.default_rng(1)
    for at in (0, 2, 9, 15):
        tokens = rng.integers(0, VOCAB, at + 6).tolist()
        far = apart(plain[which].logits(tokens, {at: (tokens[at] + 1) % VOCAB}), plain[which].logits(tokens))
        assert far[:at + 1].max() == 0 and far[at + 1:].min() > 2 * tol, (at, far)
