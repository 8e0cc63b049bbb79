"""The compiled kernels of the token mixers (no GPU needed): registers, and none saved before all lanes are back."""
from __future__ import annotations

import pytest

from test_build_lanes import test_no_register_saved_before_all_lanes_are_back as check_lanes
from test_build_resources import resources  # noqa: F401  (fixture)


@pytest.mark.parametrize("src", ("k_conv.hip", "k_delta.hip"))
def test_no_register_saved_early(src):
    check_lanes(src)


def test_scan_holds_two_workgroups_per_cu(resources):  # noqa: F811
    """Two workgroups of a compute unit hide each other's barriers: two waves a SIMD, two shares of LDS."""
    figs = [v for k, v in resources.items() if "delta_scan_kernel" in k]
    assert figs and all(f["occupancy"] >= 2 and 2 * f["lds"] <= 160 * 1024 for f in figs)
