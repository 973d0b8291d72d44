"""Compiled code of the kernels that read other lanes' registers: never in a loop
that lanes leave one by one. A lane that has left keeps its register's value only as long
as the compiler leaves the register alone: a copy or a reload inside such a loop runs
without that lane.

In the assembly a loop of that kind takes lanes out of exec in front of its back edge
(s_andn2 exec, exec); one that the whole wave leaves branches on a scalar condition."""
import re

import pytest

from asm_util import assembly, kernels, no_hipcc

pytestmark = pytest.mark.skipif(no_hipcc(), reason="no hipcc")
SOURCES = ["combine.hip", "dispatch.hip"]


def _kernels(asm):
    """{name: (instructions of each basic block, successors of each)}."""
    out = {}  # a block while it is read: [lines, labels of its branches, whether the next follows]
    for name, body in kernels(asm).items():
        blocks, at = [[[], [], True]], {}
        for line in (s.split(";")[0].strip() for s in body.splitlines()):
            label = re.match(r"(\.LBB\w+):", line)
            if label:
                blocks.append([[], [], True])
                at[label.group(1)] = len(blocks) - 1
            elif line and not line.startswith("."):
                blocks[-1][0].append(line)
                branch = re.match(r"s_c?branch\w*\s+(\.LBB\w+)", line)
                if branch:
                    blocks[-1][1].append(branch.group(1))
                if branch or line.startswith("s_endpgm"):
                    blocks[-1][2] = not line.startswith(("s_branch", "s_endpgm"))
                    blocks.append([[], [], True])
        succ = [{at[b] for b in targets} | ({i + 1} if falls and i + 1 < len(blocks) else set())
                for i, (_, targets, falls) in enumerate(blocks)]
        out[name] = [b[0] for b in blocks], succ
    return out


def _loops(succ):
    """(header, latch, blocks) of every back edge to a block that dominates its source."""
    n = len(succ)
    pred = [{j for j in range(n) if i in succ[j]} for i in range(n)]
    reach, todo = set(), [0]
    while todo:
        i = todo.pop()
        if i not in reach:
            reach.add(i)
            todo += succ[i]
    dom = {i: {0} if i == 0 else set(reach) for i in reach}
    changed = True
    while changed:
        changed = False
        for i in sorted(reach - {0}):
            new = set.intersection(*(dom[p] for p in pred[i] & reach)) | {i}
            if new != dom[i]:
                dom[i], changed = new, True
    for latch in reach:
        for head in succ[latch] & dom[latch]:
            body, todo = {head}, [latch]
            while todo:
                i = todo.pop()
                if i not in body:
                    body.add(i)
                    todo += pred[i] & reach
            yield head, latch, body



def bad_loops(asm):
    found = []
    for name, (lines, succ) in _kernels(asm).items():
        for head, latch, body in _loops(succ):
            # the latch itself, or the block in front of a latch that only branches
            tail = lines[latch] if len(lines[latch]) > 1 else sum(
                (lines[i] for i in body if succ[i] & {latch}), [])
            if any(line.startswith("s_andn2_b64 exec, exec") for line in tail) and any(
                    line.startswith("v_readlane_b32") for i in body for line in lines[i]):
                found.append((name, head))
    return found


LOOP = """_Zk:
%bb.0:
	s_mov_b64 s[0:1], 0
.LBB0_1:
	{read}
	v_cmp_le_i32_e32 vcc, s4, v1
	{latch}
%bb.2:
	s_endpgm
.Lfunc_end0:
"""
PER_LANE = "s_andn2_b64 exec, exec, s[0:1]\n\ts_cbranch_execnz .LBB0_1"
WHOLE = "s_cbranch_vccz .LBB0_1"


@pytest.mark.parametrize("read,latch,bad", [
    ("v_readlane_b32 s2, v3, s4", PER_LANE, True), ("v_readlane_b32 s2, v3, s4", WHOLE, False),
    ("v_add_u32_e32 v3, 1, v3", PER_LANE, False),
    ("v_readlane_b32 s2, v3, s4",
     "s_andn2_b64 exec, exec, s[0:1]\n\ts_cbranch_execz .LBB0_3\n\ts_branch .LBB0_1\n.LBB0_3:", True)])
def test_loops_are_told_apart(read, latch, bad):
    assert bool(bad_loops(LOOP.format(read=read, latch=latch))) == bad


@pytest.mark.parametrize("src", SOURCES)
def test_lanes_are_read_by_whole_waves(src):
    asm = assembly(src)
    assert "v_readlane_b32" in asm
    bad = bad_loops(asm)
    assert not bad, (bad[:4], len(bad))
