"""Counted memory waits in the compiled attention kernels that share keys (no GPU needed).

The 8-bit forms bring steps of K, V and scales to LDS with direct loads, several steps
ahead, and before a step is widened to bf16 they wait with s_waitcnt vmcnt(L) or vmcnt(2 L),
L being the direct loads of a step and one or two later steps being on their way.  That is
right only if every step has exactly L direct loads (fewer, and the wait would let the step
itself still be on its way), and if the compiler leaves the reads of the step behind the
wait: each 16-byte piece is read once from LDS and stored twice, widened.  This test reads
the device assembly the build writes and checks both, along every way from a wait to the
barrier that ends the turn."""
from __future__ import annotations

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_gemv_gemm_amd", "csrc")

# (head width): K or V pieces a wave brings of a step, and whether a wave brings only one of the two
BRINGS = {64: (1, True), 128: (1, False), 256: (1, False)}
RING = {64: 4, 128: 4, 256: 2}


def _blocks(body):
    """[(label, lines, labels it goes on to)] in the order of the listing."""
    blocks = [("entry", [])]
    for raw in body.split("\n"):
        line = re.sub(r"\s*;.*", "", raw.strip())
        m = re.match(r"(\.LBB\d+_\d+):", line)
        if m:
            blocks.append((m.group(1), []))
        elif line and not line.startswith("."):
            blocks[-1][1].append(line)
    out = []
    for i, (label, lines) in enumerate(blocks):
        to = [m.group(1) for m in (re.match(r"s_(?:c?branch\S*)\s+(\.LBB\d+_\d+)", x) for x in lines) if m]
        ends = any(re.match(r"s_(branch|endpgm)", x) for x in lines)
        if not ends and i + 1 < len(blocks):
            to.append(blocks[i + 1][0])
        out.append((label, lines, to))
    return out


def _kernels(text):
    """(head width, blocks) of the 8-bit kernels whose waves share keys."""
    pat = r"^(_ZN2tl\w*tree_share_kernelILi(\d+)ELb1E\w*):[^\n]*\n(.*?)^\.Lfunc_end"
    for _, width, body in re.findall(pat, text, re.S | re.M):
        yield int(width), _blocks(body)


def _is_dma(line):
    return re.match(r"(global|buffer)_load\S*", line) is not None and ("_load_lds" in line or line.endswith(" lds"))


def _counted(line):
    m = re.match(r"s_waitcnt vmcnt\((\d+)\)$", line)
    return int(m.group(1)) if m else 0


def _dma_groups(blocks):
    """Direct loads of each place that brings a step: blocks next to each other in the listing count together
    (a wave that brings K alone passes the others' blocks by)."""
    groups, last = [], -10
    for i, (_, lines, _) in enumerate(blocks):
        n = sum(_is_dma(x) for x in lines)
        if n:
            if i - last <= 2:
                groups[-1].append(n)
            else:
                groups.append([n])
            last = i
    return groups


def _ways(blocks, at, line):
    """Every way from line `line` of block `at` to the next barrier: the set of (16-byte LDS reads, writes, direct loads)."""
    index = {label: i for i, (label, _, _) in enumerate(blocks)}
    found, seen, todo = set(), set(), [(at, line, 0, 0, 0)]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        b, j, r, w, d = state
        assert r < 64 and w < 64 and d < 64, "a loop without a barrier"
        _, lines, to = blocks[b]
        for x in lines[j:]:
            if x.startswith("s_barrier") or x.startswith("s_endpgm"):
                found.add((r, w, d))
                break
            r += x.startswith("ds_read_b128")
            w += x.startswith("ds_write_b128")
            d += _is_dma(x)
        else:
            todo += [(index[t], 0, r, w, d) for t in to]
    return found


def _faults(width, blocks):
    """What is wrong with a kernel's counted waits."""
    mine, either = BRINGS[width]
    loads = (1 if either else 2) * mine + 1                # of a wave, for one step
    bad = []
    for g in _dma_groups(blocks):
        if (either and g != [mine, mine, 1]) or (not either and sum(g) != loads):
            bad.append(f"a step brought by direct loads {g}, not {loads}")
    waits = [(i, j, _counted(x)) for i, (_, lines, _) in enumerate(blocks) for j, x in enumerate(lines) if _counted(x)]
    waits = [x for x in waits if x[2] > 1]                 # those of one load are the compiler's own
    if {n for _, _, n in waits} != ({loads, 2 * loads} if RING[width] == 4 else set()):
        bad.append(f"waits for {sorted({n for _, _, n in waits})} with {loads} loads a step")
    for i, j, n in waits:
        for r, w, d in _ways(blocks, i, j + 1):
            if 2 * r != w or d:
                bad.append(f"vmcnt({n}): {r} pieces read, {w} written, {d} direct loads before the barrier")
        if not any(w for _, w, _ in _ways(blocks, i, j + 1)):
            bad.append(f"vmcnt({n}): nothing is widened behind it")
    return bad


@pytest.fixture(scope="module")
def listing():
    from quantized_gemv_gemm_amd import _build
    path = _build.asm_path("k_tree.hip")
    newest = max(os.path.getmtime(os.path.join(CSRC, f)) for f in os.listdir(CSRC))
    if not os.path.exists(path) or os.path.getmtime(path) < newest:
        _build.build()
    with open(path) as f:
        return f.read()


def test_the_sources_count_what_is_checked(listing):
    with open(os.path.join(CSRC, "k_tree.hip")) as f:
        src = f.read()
    assert "static constexpr int ring = D == 256 && E4M3 ? 2 : 4;" in src
    assert "static constexpr int loads = (halves ? 1 : 2) * mine + (E4M3 ? 1 : 0);" in src
    assert sorted(w for w, _ in _kernels(listing)) == [64, 128, 256]


def test_counted_waits_cover_a_step(listing):
    for width, blocks in _kernels(listing):
        assert len(_dma_groups(blocks)) >= 3
        assert _faults(width, blocks) == [], width


FAKE = """_ZN2tl1_tree_share_kernelILi128ELb1ELi2EEEv: ; @x
	s_cbranch_scc1 .LBB0_3
.LBB0_1:
	global_load_lds_dwordx4 v[4:5], off
	global_load_lds_dwordx4 v[4:5], off offset:16
	global_load_lds_dword v[6:7], off
	s_cbranch_scc1 .LBB0_4
.LBB0_2:
	s_waitcnt vmcnt(6)
	s_branch .LBB0_5
.LBB0_3:
	v_mov_b32_e32 v1, v2
.LBB0_4:
	s_waitcnt vmcnt(3)
.LBB0_5:
	ds_read_b128 v[8:11], v1
	ds_write_b128 v2, v[8:11]
	ds_write_b128 v2, v[8:11] offset:1024
	ds_read_b128 v[12:15], v1 offset:16
	ds_write_b128 v3, v[12:15]
	ds_write_b128 v3, v[12:15] offset:512
	s_waitcnt lgkmcnt(0)
	s_barrier
	s_endpgm
.Lfunc_end0:
"""


def _planted(old, new):
    text = FAKE.replace(old, new, 1)
    assert text != FAKE or old == new
    ((width, blocks),) = list(_kernels(text))
    return _faults(width, blocks)


def test_checker_flags_planted_faults():
    read = "\tds_read_b128 v[8:11], v1\n"
    assert _planted("", "") == []
    assert _planted("\tglobal_load_lds_dword v[6:7], off\n", "")       # a step of two loads, waits for three
    assert _planted("vmcnt(6)", "vmcnt(5)")
    assert _planted("\ts_waitcnt vmcnt(6)\n", read + "\ts_waitcnt vmcnt(6)\n") == []
    moved = FAKE.replace(read, "", 1).replace("\ts_waitcnt vmcnt(3)\n", read + "\ts_waitcnt vmcnt(3)\n", 1)
    ((width, blocks),) = list(_kernels(moved))                         # a piece read before the wait
    assert any("1 pieces read, 4 written" in x for x in _faults(width, blocks))
