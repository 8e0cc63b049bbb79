"""Corners of the token mixers' contracts on the GPU: the longest request when it is not named."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.mixers as ref
from gpu_common import announce, to_dev
from test_gpu_mixers import Step, _check_delta, _delta_inputs, dev, f64, tl, torch  # noqa: F401

pytestmark = pytest.mark.gpu


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
