"""Waits inside assembly along every way through the code: the rule of test_asm_waits.py (a memory
instruction reads a scalar register at the earliest five wait states after a vector instruction wrote
it, m0 one after its write), followed over branches, taken and not, back to a loop's head included.

Of each register that was written lately, the fewest wait states that any way from its write needs
are kept at each instruction; an instruction that a way reaches with fewer is gone through again."""
import pathlib
import re
import shutil
import subprocess

import pytest

from test_asm_waits import LIBRARY, OBJDUMP, STATES, scalars


def effects(line):
    """(registers read by a memory instruction, states it lasts, {register: states its write needs},
    registers whose wait ends)."""
    op, _, rest = line.partition(" ")
    parts = [x.strip() for x in re.split(r",(?![^\[]*\])", rest)]
    reads, wrote, ended = frozenset(), {}, frozenset()
    if op.startswith(("buffer_", "global_", "flat_", "scratch_")):
        reads = frozenset(scalars(rest) | ({124} if rest.endswith("lds") else set()))
    lasts = int(rest, 0) + 1 if op == "s_nop" else 1
    if op.startswith(("v_readfirstlane", "v_readlane")) or op.startswith("v_cmp") and not op.startswith("v_cmpx"):
        wrote = {r: STATES for r in scalars(parts[0])}
    elif op.startswith(("v_add_co", "v_sub_co", "v_addc_co", "v_subb_co", "v_mad_u64", "v_mad_i64", "v_div_scale")):
        wrote = {r: STATES for r in scalars(parts[1])}
    elif op.startswith("s_") and not op.startswith(("s_cmp", "s_bitcmp", "s_nop", "s_waitcnt", "s_barrier", "s_branch",
                                                    "s_cbranch", "s_setprio", "s_endpgm")):
        ended = frozenset(scalars(parts[0]))
        wrote = {124: 1} if 124 in ended else {}
    return reads, lasts, wrote, ended


def hazards(code):
    """code: [(address, instruction, branch target or None)].  Reads that come too soon on some way."""
    index = {a: i for i, (a, _, _) in enumerate(code)}
    fx = [effects(line) for _, line, _ in code]
    left = [None] * len(code)                  # register -> wait states that it still needs here
    found, todo = set(), [(0, {})]
    while todo:
        i, state = todo.pop()
        while i < len(code):
            seen = left[i]
            if seen is None:
                left[i] = dict(state)
            else:
                more = {r: n for r, n in state.items() if n > seen.get(r, 0)}
                if not more:
                    break
                seen.update(more)
                state = dict(seen)
            _, line, target = code[i]
            reads, lasts, wrote, ended = fx[i]
            found |= {(code[i][0], line, r, state[r]) for r in reads if state.get(r, 0) > 0}
            state = {r: n - lasts for r, n in state.items() if n > lasts and r not in ended}
            state.update(wrote)
            if target is not None and target in index:
                todo.append((index[target], dict(state)))
            if line.startswith(("s_branch", "s_endpgm", "s_setpc")):
                break
            i += 1
    return sorted(found)


def parse(text):
    """[(kernel, code)] of a disassembly with addresses."""
    out = []
    for kernel in re.split(r"^[0-9a-f]+ <(?=\S+>:$)", text, flags=re.M)[1:]:
        name, *lines = kernel.split("\n")
        start, code = None, []
        for x in lines:
            m = re.match(r"\s+(\S.*?)\s*// ([0-9A-F]+):(.*)$", x)
            if not m:
                continue
            line, address = re.sub(r"\s+", " ", m.group(1)).strip(), int(m.group(2), 16)
            start = address if start is None else start
            to = re.search(r"<[^>]*\+0x([0-9a-f]+)>", m.group(3)) if line.startswith(("s_branch", "s_cbranch")) else None
            if line.startswith(("s_branch", "s_cbranch")):
                assert to or m.group(3).rstrip().endswith(">"), x
            target = None if not line.startswith(("s_branch", "s_cbranch")) else start + (int(to.group(1), 16) if to else 0)
            code.append((address, line, target))
        out.append((name, code))
    return out


def test_the_rule_itself():
    read = "buffer_load_dwordx4 v1, s[24:27], s42 offen lds"
    first, m0 = "v_readfirstlane_b32 s26, v1", "s_mov_b32 m0, s9"

    def code(lines, **to):
        return [(4 * i, x, to.get(f"at{i}")) for i, x in enumerate(lines)]

    assert hazards(code([first, "s_mov_b32 s0, s1", m0, "s_nop 0", read]))
    assert not hazards(code([first, m0, "s_nop 3", read]))
    assert hazards(code([m0, read])) and not hazards(code([m0, "s_nop 0", read]))
    # written at the loop's end, read at its head
    loop = ["s_mov_b32 s0, s1", m0, "s_nop 0", read, "s_nop 4", first, "s_cbranch_scc0 65529", "s_endpgm"]
    assert hazards(code(loop, at6=4)) and not hazards(code(loop))
    # over a branch that jumps past the wait
    jump = [first, "s_cbranch_scc0 2", "s_nop 4", m0, "s_nop 0", read, "s_endpgm"]
    assert hazards(code(jump, at1=12)) and not hazards(code(jump))
    # the way with the wait comes first: the other is still looked at
    both = ["s_cbranch_scc0 3", first, "s_nop 4", "s_branch 1", first, m0, "s_nop 0", read, "s_endpgm"]
    assert hazards(code(both, at0=16, at3=20))


def test_no_way_reads_too_soon(tmp_path):
    if not OBJDUMP.exists() or not LIBRARY.exists():
        pytest.skip("needs the library and a disassembler")
    shutil.copy(LIBRARY, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", LIBRARY.name], cwd=tmp_path, check=True, capture_output=True)
    branches, found = 0, []
    for path in sorted(tmp_path.glob("*gfx950")):
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", path], check=True, capture_output=True, text=True).stdout
        for name, code in parse(text):
            branches += sum(t is not None for _, _, t in code)
            addresses = {a for a, _, _ in code}
            assert all(t is None or t in addresses for _, _, t in code), name
            found += [(name, *x) for x in hazards(code)]
    assert branches > 1000
    assert not found, (len(found), found[:3])
