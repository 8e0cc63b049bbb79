"""Corners of the token mixers' contracts on the GPU: keys that are not finite in an 8-bit cache and the
longest request when it is not named."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.mixers as ref
import oracle.speculative as spec
from gpu_common import announce, to_dev
from test_gpu_mixers import Step, _check_delta, _delta_inputs, bf16_dev, bits, dev, f64, tl, torch  # noqa: F401

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
