"""Registers saved before all lanes are back, in the compiled kernels (no GPU needed).

Where lanes that parted at a branch meet again, a block begins with the instruction that
switches the lanes that stayed away on again (s_or_b64 exec, exec, ...).  The compiler has
been seen to put a register's move to another place (v_mov, v_accvgpr_write) before it: the
value then lacks the lanes that were away, and what is computed from it later, a store's
address say, is wrong in them.  It happened in a kernel that needs nearly all registers, and
went away with the branch.  This test reads the device assembly the build writes: no block
may have nothing but such moves before that instruction."""
from __future__ import annotations

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_gemv_gemm_amd", "csrc")
SOURCES = ("k_gemv.hip", "k_gemm.hip", "k_kv.hip", "k_step.hip", "k_tree.hip", "k_verify.hip")

MOVE = re.compile(r"v_(mov_b(32|64)\S* v\S+ v|accvgpr_)")
END = re.compile(r"s_(cbranch|branch|endpgm)|\S*saveexec|s_(and|andn2|xor|mov)_b64 exec")


def _early_moves(text):
    """(block, moves) of every block that has only moves of vector registers before its lanes are back."""
    found, label, vector = [], None, []
    for raw in text.split("\n"):
        line = re.sub(r"\s*;.*", "", raw.strip())
        if re.match(r"\.LBB\d+_\d+:", line):
            label, vector = line, []
        elif label is None or not line:
            continue
        elif line.startswith("s_or_b64 exec, exec"):
            if vector and all(MOVE.match(v) for v in vector):
                found.append((label, vector))
            label = None
        elif END.match(line):
            label = None
        elif re.match(r"v_(?!writelane|readlane|readfirstlane)|ds_|global_|buffer_", line):
            vector.append(line)
    return found


@pytest.mark.parametrize("src", SOURCES)
def test_no_register_saved_before_all_lanes_are_back(src):
    from quantized_gemv_gemm_amd import _build
    path = _build.asm_path(src)
    newest = max(os.path.getmtime(os.path.join(CSRC, f)) for f in os.listdir(CSRC))
    if not os.path.exists(path) or os.path.getmtime(path) < newest:
        _build.build()
    with open(path) as f:
        assert _early_moves(f.read()) == []


def test_a_planted_early_move_is_found():
    bad = [".LBB9_140:   ; in Loop", "\tv_accvgpr_write_b32 a169, v16", "\ts_mov_b64 s[78:79], s[36:37]",
           "\ts_or_b64 exec, exec, s[2:3]", "\tv_mul_lo_u32 v2, s35, v12"]
    good = [bad[0], bad[2], bad[3], bad[1], bad[4]]
    body = [".LBB0_37:", "\tv_sub_f32_e32 v4, v28, v45", "\tv_mov_b32_e32 v5, v4", "\ts_or_b64 exec, exec, s[2:3]"]
    assert [b for b, _ in _early_moves("\n".join(bad))] == [".LBB9_140:"]
    assert _early_moves("\n".join(good)) == [] and _early_moves("\n".join(body)) == []
