"""Corners of the speculative-decoding operators without a GPU: views whose tokens overlap,
sizes at the edge of what the kernels' integers hold, and the plain definitions beside them."""
from __future__ import annotations

import ctypes
import json
import os
import re
from fractions import Fraction

import numpy as np
import pytest

import oracle.speculative as ref
import quantized_gemv_gemm_amd as tl

pytestmark = pytest.mark.skipif(not os.path.exists(tl.LIB_PATH), reason="libtl.so not built")


# --------------------------------------------------------------------------- rows of q, k and v
def test_rows_closer_than_a_row_are_refused():
    """Tokens that share elements (a broadcast token, a sliding window) have no distance the kernels take."""
    torch = pytest.importorskip("torch")
    one = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    flat = torch.zeros(40 * 128, dtype=torch.bfloat16)
    for view in (one.expand(8, 4, 128), flat.as_strided((8, 4, 128), (128, 128, 1)),
                 flat.as_strided((8, 4, 128), (4 * 128 - 8, 128, 1)), one[:, :1].expand(2, 1, 128)):
        for name in ("q", "k", "v"):
            with pytest.raises(ValueError, match=name):
                tl._rows(view, name, -1)


def test_rows_give_their_own_distance():
    torch = pytest.importorskip("torch")
    wide = torch.zeros((6, 20 * 64), dtype=torch.bfloat16)
    assert tl._rows(wide.unflatten(1, (20, 64)), "q", -1) == (wide.data_ptr(), 20 * 64)
    part = wide[:, 128:128 + 4 * 64].unflatten(1, (4, 64))
    assert tl._rows(part, "k", -1) == (part.data_ptr(), 20 * 64)
    assert tl._rows(part[::3], "k", -1)[1] == 60 * 64
    # one token or none: whatever the stride says, nothing is stepped over
    assert tl._rows(part[:1].expand(1, 4, 64), "k", -1)[1] == 4 * 64
    assert tl._rows(wide.as_strided((1, 4, 64), (0, 64, 1)), "k", -1)[1] == 4 * 64
    assert tl._rows(part[:0], "k", -1)[1] == 4 * 64
    # one head: the distance of heads does not matter
    assert tl._rows(wide.as_strided((3, 1, 64), (128, 7, 1)), "v", -1)[1] == 128


# --------------------------------------------------------------------------- sizes
def attention_status(T=1, H=1, G=1, D=64, block=16, width=4, R=1):
    """Status of a call without a workspace: 7 if nothing before it is refused."""
    P = lambda n: ctypes.c_void_p((n + 1) << 40)
    return tl.lib().tl_tree_attention(P(0), H * G * D, T, H, G, D, P(1), P(2), None, None, tl.TL_BF16, 9, block, P(3), width,
                                      R, P(4), P(5), None, 0.1, 1, P(6), None, None, 0, None)


@pytest.mark.parametrize("block", [16, 64, 4096])
def test_attention_positions_stay_in_31_bits(block):
    """Keys are counted in 32 bits, up to 64 tiles past the last one: wider tables would give negative positions."""
    most = ((1 << 31) - 4096) // block
    assert attention_status(block=block, width=most) == 7
    assert attention_status(block=block, width=most + 1) == 2


# --------------------------------------------------------------------------- the plain definitions, by hand
def test_plan_beyond_capacity_by_hand():
    """Request 1's tokens pass the capacity: it and the later ones with tokens or a need of pages are not served."""
    table = np.zeros((5, 3), dtype=np.int64)
    got = ref.step_plan(np.array([14, 10, 16, 20, 8]), np.array([3, 8, 0, 0, 1]), np.array([1, 1, 1, 1, 1]), table,
                        np.array([9, 8, 7, 6]), 0, 10, 16, np.array([-1, 0, 0] + [-1, 0, 1, 2, 3, 4, 5]))
    q_start, kv, slots, pos, mask, owned, head, out = got
    assert q_start.tolist() == [0, 3, 10, 10, 10, 10]
    assert kv.tolist() == [17, 0, 16, 0, 0] and owned.tolist() == [2, 1, 1, 1, 1] and head == 1
    assert out[0].tolist() == [0, 9, 0] and not out[1:].any()
    assert slots.tolist() == [14, 15, 9 * 16] + [-1] * 7 and mask[9] == 127 and pos[9] == 16


def test_commit_of_a_path_cut_short_by_hand():
    """Five accepted nodes, three of them on the path; a prompt of 100 tokens needs none."""
    moves, ctx = ref.commit_moves([5, 100], np.array([[0, 2, 3], [-1, -1, -1]]), [15, 4], [25, 104], np.zeros((2, 8)), 3, 16)
    assert moves == [(0, 0, 1, 0, 0), (0, 0, 2, 0, 1)] and ctx.tolist() == [18, 104]


def test_attention_kernels_fit_lds_at_the_most_requests():
    """The compiler's count of static LDS stays within what the sources keep free for it beside the ring
    and the prefix sums of 4096 requests."""
    from quantized_gemv_gemm_amd import _build
    with open(_build.RESOURCES) as f:
        figs = {k: v["lds"] for k, v in json.load(f).items() if "tree_split_kernel" in k or "tree_share_kernel" in k}
    with open(os.path.join(_build.CSRC, "tl_internal.h")) as f:
        free = int(re.search(r"kStaticLds = (\d+);", f.read()).group(1))
    assert len(figs) > 10 and max(figs.values()) <= free


@pytest.mark.parametrize("H,T,G,R,block", [(1, 1 << 17, 16, 4096, 64), (8, 65536, 8, 1, 16), (64, 4096, 64, 64, 4096),
                                           (65536, 16, 1, 7, 128)])
def test_attention_units_stay_in_31_bits(H, T, G, R, block):
    """The documented limit, H (T G / 16 + R) (width block / 128 + 1) < 2^31, at its two sides."""
    def units(width):
        return Fraction(H) * (Fraction(T * G, 16) + R) * (Fraction(width * block, 128) + 1)
    lo, hi = 0, ((1 << 31) - 4096) // block + 1
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if units(mid) < 1 << 31 else (lo, mid)
    assert attention_status(T=T, H=H, G=G, R=R, block=block, width=lo) == 7
    assert attention_status(T=T, H=H, G=G, R=R, block=block, width=hi) == 2


def test_offset_refuses_caches_beyond_the_limit():
    """pages * H * block * D stays within 2^50: past it an offset would not fit its type."""
    L = tl.lib()
    page = (1 << 50) // (65536 * 4096 * 256) - 1
    assert L.tl_kv_offset(0, tl.TL_E4M3, 65536, 256, 4096, page, 65535, 4095, 255) == (1 << 50) - 1
    for far in (page + 1, 1 << 30, (1 << 31) - 1):
        assert L.tl_kv_offset(0, tl.TL_E4M3, 65536, 256, 4096, far, 65535, 4095, 255) == -1
    assert L.tl_kv_offset(1, tl.TL_BF16, 1, 64, 16, (1 << 31) - 2, 0, 15, 63) == ((1 << 31) - 1) * 1024 - 1
