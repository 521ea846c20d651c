"""The shared-memory reads that the tile kernels of FP8 with group scales ask for ahead of their use: in the assembly
that hipcc writes for them, nothing touches a read's registers before the wait for it (CPU).  The compiler takes such
a read's registers as written at once; a copy or a spill of one that is still on its way would be wrong."""
import os
import re
import subprocess

import pytest

from tensor_transformer_mlp_02_amd import build as b

REG = re.compile(r"\bv\[(\d+):(\d+)\]|\bv(\d+)\b")


def registers(text):
    out = set()
    for m in REG.finditer(text):
        out |= set(range(int(m.group(1)), int(m.group(2)) + 1)) if m.group(1) else {int(m.group(3))}
    return out


def kernels(lines):
    """Each kernel's basic blocks: label -> ([(line, op, operands, in inline assembly)], labels that may follow)."""
    inline, blocks, label = False, {}, None
    for n, line in enumerate(lines, 1):
        if "#ASMSTART" in line:
            inline = True
        if "#ASMEND" in line:
            inline = False
        text = line.split(";")[0].strip()
        start = re.match(r"^([^\s]+):$", text)
        if start:
            if not text.startswith("."):         # the next kernel
                if blocks:
                    yield blocks
                blocks = {}
            elif label is not None and blocks and not blocks[label][2]:
                blocks[label][1].append(start.group(1))
            label = start.group(1)
            blocks[label] = ([], [], [])         # the last: whether it has ended
            continue
        if label is None or not text or text.startswith("."):
            continue
        op, _, rest = text.partition(" ")
        if op in ("s_branch", "s_endpgm") or op.startswith("s_cbranch"):
            if op != "s_endpgm":
                blocks[label][1].append(rest.strip())
            if op.startswith("s_cbranch"):       # what follows is a block of its own
                follow = f"{label}+{n}"
                blocks[label][1].append(follow)
                blocks[label][2].append(n)
                label = follow
                blocks[label] = ([], [], [])
            else:
                blocks[label][2].append(n)
            continue
        if not blocks[label][2]:
            blocks[label][0].append((n, op, rest, inline))
    if blocks:
        yield blocks


def touched_in_flight(lines):
    """(reads seen, offending lines) of a listing, along every path; reads count where they stand in inline assembly."""
    reads, bad = set(), set()
    for blocks in kernels(lines):
        before = {next(iter(blocks)): frozenset()}
        todo = list(before)
        while todo:
            label = todo.pop()
            on_the_way = set(before[label])
            for n, op, rest, inline in blocks[label][0]:
                if op.startswith("ds_read") and inline:
                    to, _, address = rest.partition(",")
                    if registers(to) & on_the_way or registers(address) & on_the_way:
                        bad.add((n, f"{op} {rest}"))
                    on_the_way |= registers(to)
                    reads.add(n)
                elif op == "s_waitcnt" and "lgkmcnt(0)" in rest:
                    on_the_way = set()
                elif registers(rest) & on_the_way:
                    bad.add((n, f"{op} {rest}"))
            for follow in blocks[label][1]:
                if follow not in blocks:
                    continue
                seen = before.get(follow)
                if seen is None or not on_the_way <= seen:
                    before[follow] = frozenset(on_the_way | (seen or frozenset()))
                    todo.append(follow)
    return len(reads), sorted(bad)


def test_the_check_sees_a_copy():
    ask = ["k:", ";;#ASMSTART", "ds_read_b128 v[4:7], v1 offset:16", ";;#ASMEND"]
    wait = [";;#ASMSTART", "s_waitcnt lgkmcnt(0)", ";;#ASMEND", "v_mov_b32 v9, v5"]
    assert touched_in_flight(ask + ["v_add_u32 v8, v2, v3"] + wait) == (1, [])
    assert touched_in_flight(ask + ["v_mov_b32 v9, v5"] + wait)[1] == [(5, "v_mov_b32 v9, v5")]
    assert touched_in_flight(ask + ["scratch_store_dwordx4 off, v[4:7], off"] + wait)[1]
    assert touched_in_flight(ask + [";;#ASMSTART", "ds_read_b32 v4, v2", ";;#ASMEND"] + wait)[1]
    # along a branch, and round a loop
    assert touched_in_flight(ask + ["s_branch .L2", ".L1:", "v_mov_b32 v9, v5", "s_endpgm", ".L2:"] + wait) == (1, [])
    assert touched_in_flight(ask + ["s_cbranch_scc1 .L2"] + wait + ["s_endpgm", ".L2:", "v_mov_b32 v9, v5"])[1]
    assert touched_in_flight(["k:", ".L1:", "v_mov_b32 v9, v5", *ask[1:], "s_cbranch_scc1 .L1", "s_endpgm"])[1]
    assert touched_in_flight(["k:", ".L1:", "v_mov_b32 v9, v5", *ask[1:], *wait, "s_cbranch_scc1 .L1", "s_endpgm"]) == (1, [])


@pytest.mark.skipif(not os.path.exists(b.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source", ["fp8g_gemm.hip", "fp8g_gemm32.hip", "fp8g_glu.hip"])
def test_nothing_touches_a_read_on_its_way(source, tmp_path):
    out = tmp_path / "listing.s"
    flags = [f for f in b.FLAGS if f != "-Wall"]
    subprocess.run([b.HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(b.CSRC, source), "-o", str(out)], check=True,
                   capture_output=True)
    reads, bad = touched_in_flight(out.read_text().splitlines())
    assert reads > 300 and not bad, bad[:5]
