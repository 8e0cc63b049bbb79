"""The compiled kernels of the token mixers (no GPU needed): registers, and none saved before all lanes are back."""
from __future__ import annotations

import pytest

from test_build_lanes import test_no_register_saved_before_all_lanes_are_back as check_lanes
from test_build_resources import resources  # noqa: F401  (fixture)


@pytest.mark.parametrize("src", ("k_conv.hip", "k_delta.hip"))
def test_no_register_saved_early(src):
    check_lanes(src)


@pytest.mark.parametrize("kernel,waves,groups", [("delta_scan_kernel", 2, 1), ("delta_chunk_kernel", 4, 2), ("delta_prep_kernel", 2, 2),
                                                 ("delta_step_kernel", 5, 5)])
def test_nothing_spills(resources, kernel, waves, groups):  # noqa: F811
    """Waves on a SIMD, workgroups whose LDS a compute unit holds, and no scratch memory."""
    figs = [v for k, v in resources.items() if kernel in k]
    assert len(figs) >= 2
    for f in figs:
        assert f["occupancy"] >= waves and groups * f["lds"] <= 160 * 1024 and f["scratch"] == 0, f
