"""Corners of the token mixers' contracts on the GPU: keys that are not finite in an 8-bit cache, the longest request when it
is not named, accepted counts past a tree's tokens."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.mixers as ref
import oracle.speculative as spec
from gpu_common import announce, to_dev
from test_gpu_mixers import STATE_TOL, _check_delta, _delta_inputs, Step, bf16_dev, bits, dev, f64, tl, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("D,rot", [(64, 0), (128, 64), (256, 256)])
def test_a_key_that_is_not_finite_shows_in_an_8bit_cache(tl, torch, D, rot, what):  # noqa: F811
    """The norm spreads one such element over its row: scale and values read NaN, as the rows of a bfloat16 cache and of q
    do, and no other token's or head's row changes."""
    announce(f"normed write of a {what}, D={D}")
    d, rng, T, H, block = dev(), np.random.default_rng(D), 21, 2, 16
    x = spec.bf16(rng.standard_normal((T, 3 * H, D)))
    cs = to_dev(rng.uniform(-1, 1, (64, rot)).astype(np.float32), d) if rot else None
    slots, pos = to_dev(np.arange(T) + 3, d), to_dev(rng.integers(0, 64, T).astype(np.int32), d)

    def write(x, dtype):
        xd = bf16_dev(x, d)
        cache = tl.kv_cache(3, H, block, D, dtype=dtype, device=d)
        q = tl.kv_write_norm(xd[:, H:2 * H], xd[:, 2 * H:], slots, *cache[:2], k_scale=cache[2], v_scale=cache[3], q=xd[:, :H],
                             positions=pos if rot else None, cos_sin=cs)
        torch.cuda.synchronize()
        return (q, *cache)

    bad = x.copy()
    for t, head, at in ((2, 1, 5), (17, 0, D - 1)):
        bad[t, H + head, at] = bad[t, head, at] = what
    for dtype in (torch.float8_e4m3fn, torch.bfloat16):
        good, got = write(x, dtype), write(bad, dtype)
        es = 1 if dtype is torch.float8_e4m3fn else 2
        k_at, rows = spec.offsets("k", es, block, D), bits(got[1]).reshape(3, H, -1)
        same = bits(good[1]).reshape(3, H, -1).copy()
        for t, head, _ in ((2, 1, 5), (17, 0, D - 1)):
            page, i = divmod(t + 3, block)
            row = rows[page, head, k_at[i]]
            if es == 1:
                assert np.isnan(got[3][page, head, i].item()) and np.isnan(spec.e4m3_value(row)).all(), (t, row)
            else:
                assert np.isnan((row.view(np.uint16).astype(np.uint32) << 16).view(np.float32)).any()
            assert torch.isnan(got[0][t, head]).any()
            same[page, head, k_at[i]] = row
            if es == 1:
                good[3][page, head, i] = got[3][page, head, i]
        np.testing.assert_array_equal(rows, same)
        np.testing.assert_array_equal(bits(got[2]), bits(good[2]))
        if es == 1:
            np.testing.assert_array_equal(bits(got[3]), bits(good[3]))
            np.testing.assert_array_equal(bits(got[4]), bits(good[4]))


@pytest.mark.parametrize("lens,kernel", [([1] * 63 + [300], "delta_scan"), ([300] + [1] * 63, "delta_scan"), ([64], "delta_chunk"),
                                         ([1] * 64, "delta_step"), ([2, 0, 3], "delta_step"), ([20, 1, 40], "delta_chunk")], ids=str)
def test_delta_rule_without_max_nodes(tl, torch, lens, kernel):  # noqa: F811
    """The longest request is not named: a prompt beside single tokens does not go token by token."""
    announce(f"delta_rule without max_nodes, {len(lens)} requests of up to {max(lens)}")
    d, rng = dev(), np.random.default_rng(len(lens))
    s = Step(np.array(lens), rng, behind=0)
    plain, given, _, state = _delta_inputs(s, 1, 2, 64, 32, rng, False, d)
    stated = to_dev(state, d)
    got = tl.delta_rule(*given, *s.dev(d), stated)
    torch.cuda.synchronize()
    assert tl.last_kernel_name() == kernel
    want, after, size = ref.delta_rule(*plain, s.q_start, s.kv_lens, s.slots, state.astype(np.float64), None, 0.125,
                                       np.zeros((s.T, 2, 32)))
    _check_delta(f64(got), stated.cpu().numpy(), want, after, size, state, s.T)


def test_commit_of_a_path_longer_than_the_tree(tl, torch):  # noqa: F811
    """accepted counts entries of the path up to its width; those that name no token are skipped, and the others are taken,
    also where there are more entries than the tree has tokens."""
    announce("commit of a path longer than the tree")
    d, rng = dev(), np.random.default_rng(3)
    s = Step(np.array([2, 3, 1]), rng, trees=True, unserved=False)
    plain, given, _, state = _delta_inputs(s, 1, 2, 64, 32, rng, False, d)
    accepted = np.array([3, 9, 2], np.int32)
    path = np.array([[-1, 0, 1, -1, -1, 0], [0, 7, -3, 1, 1 << 30, 2], [5, 0, -1, -1, -1, -1]], np.int32)
    x, conv = spec.bf16(rng.standard_normal((s.T, 64))), spec.bf16(rng.standard_normal((s.states, 3, 64)))
    stated, convd = to_dev(state, d), bf16_dev(conv, d)
    tl.delta_commit(to_dev(accepted, d), to_dev(path, d), *s.dev(d), *given[1:], stated, x=bf16_dev(x, d), conv_state=convd)
    torch.cuda.synchronize()
    # by hand: the chains of tokens 0, 1 of request 0, of 0, 1, 2 of request 1, and of token 0 of request 2
    lens = [2, 3, 1]
    _, want, _ = ref.delta_rule(*plain, s.q_start, s.kv_lens, s.slots, state.astype(np.float64), None, 1.0,
                                np.zeros((s.T, 2, 32)))
    got = stated.cpu().numpy()
    for r in range(3):
        row, first, n = s.slots[r], s.q_start[r], lens[r]
        assert np.linalg.norm(got[row] - want[row]) <= STATE_TOL * np.linalg.norm(want[row]), r
        old = np.zeros((3, 64)) if s.kv_lens[r] <= n else conv[row]
        np.testing.assert_array_equal(f64(convd[row]), np.concatenate([old, x[first:first + n]])[-3:])
    by_oracle, _ = ref.delta_commit(accepted, path, s.q_start, s.kv_lens, s.slots, *plain[1:], state.astype(np.float64), x, conv)
    np.testing.assert_allclose(by_oracle, want, rtol=1e-12)
