"""Scalar-operand hazard scan of the gfx950 code of every kernel (CPU only).

A vector memory instruction that reads a scalar register needs five wait
states after a vector instruction that wrote it (v_readlane, v_readfirstlane,
a compare).  The compiler inserts them before its own loads, but it does not
look into inline asm: a load that goes straight into LDS and is written there
has to bring them itself, or it may take a stale descriptor or offset.  The
same goes for the one wait state between a write of m0 and a load into LDS.
This test compiles every HIP source to gfx950 assembly, as the build does, and
follows the code after each such write, across block labels and branches.
"""

import os
import re
import subprocess

import pytest

from test_isa_store_hazard import CSRC, HIPCC, ROOT, SOURCES, functions, wait_states

WINDOW = 5          # wait states from a vector write of a scalar register to a vector memory read of it
VMEM = re.compile(r"^(buffer|global|flat|scratch|tbuffer)_")


def sregs(tok):
    """Scalar registers named by one operand."""
    tok = tok.strip()
    m = re.match(r"s\[(\d+):(\d+)\]$", tok)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.match(r"s(\d+)$", tok)
    if m:
        return {int(m.group(1))}
    return {"vcc_lo": {"vcc_lo"}, "vcc_hi": {"vcc_hi"}, "vcc": {"vcc_lo", "vcc_hi"}, "m0": {"m0"}}.get(tok, set())


def operands(op):
    parts = op.split(None, 1)
    return [o.strip() for o in parts[1].split(",")] if len(parts) > 1 else []


def read_by_memory(op):
    """Scalar registers that a vector memory instruction reads."""
    out = set().union(*[sregs(t) for t in re.findall(r"\bs\[\d+:\d+\]|\bs\d+\b|\bvcc(?:_lo|_hi)?\b", op)])
    return out | {"m0"} if " lds" in op else out


def written(op):
    """Scalar registers that an instruction writes (its first operand; the
    second too, where a vector instruction has a carry or scale result)."""
    ops = operands(op)
    if not ops or re.match(r"s_(nop|waitcnt|barrier|branch|cbranch|cmp|bitcmp|endpgm|setprio|sleep|sendmsg)", op):
        return set()
    if op.startswith("s_"):
        return sregs(ops[0])
    if op.startswith("v_"):
        out = sregs(ops[0])
        if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale|v_mad_[iu]64", op) and len(ops) > 1:
            out |= sregs(ops[1])
        return out
    return set()


def scan(asm):
    problems, checked = [], 0
    for fn, (ins, labels) in functions(asm).items():
        for k, op in enumerate(ins):
            if VMEM.match(op) and " lds" in op:
                checked += 1
            to_lds_only = op.startswith("s_") and "m0" in written(op)
            if not (op.startswith("v_") and written(op)) and not to_lds_only:
                continue
            # (next instruction, wait states passed, registers still stale)
            todo, seen = [(k + 1, 0, frozenset(written(op)))], set()
            while todo:
                at, waits, live = todo.pop()
                if at >= len(ins) or not live or waits >= (1 if to_lds_only else WINDOW) or (at, waits, live) in seen:
                    continue
                seen.add((at, waits, live))
                nxt = ins[at]
                if VMEM.match(nxt):
                    if read_by_memory(nxt) & live:
                        problems.append(f"{fn}: '{op}' then, {waits} wait states later, '{nxt}'")
                        continue
                if nxt.startswith("s_endpgm"):
                    continue
                live, waits = live - written(nxt), waits + wait_states(nxt)
                m = re.match(r"s_(c?)branch\w*\s+(\.L\w+)", nxt)
                if m and m.group(2) in labels:
                    todo.append((labels[m.group(2)], waits, live))
                    if not m.group(1):
                        continue
                todo.append((at + 1, waits, live))
    return problems, checked


def test_scanner_flags_the_pattern():
    load = "\tbuffer_load_dwordx4 v3, s[28:31], s26 offen lds\n"
    asm = "\ts_mov_b32 m0, s5\n\ts_nop {nop}\n" + load + "\ts_endpgm\n"
    descriptor = "kern:\n\tv_readlane_b32 s31, v200, 7\n" + asm
    offset = "kern:\n\tv_readfirstlane_b32 s26, v1\n" + asm
    across = "kern:\n\tv_readlane_b32 s28, v200, 7\n\ts_branch .LBB0_2\n.LBB0_2:\n" + asm
    other = "kern:\n\tv_readlane_b32 s32, v200, 7\n" + asm
    again = "kern:\n\tv_readlane_b32 s26, v200, 7\n\ts_mov_b32 s26, 0\n" + asm
    for bad in (descriptor, offset, across):
        assert scan(bad.format(nop=0))[0] and not scan(bad.format(nop=3))[0]
    assert scan(descriptor.format(nop=2))[0]
    for good in (other, again):
        assert scan(good.format(nop=0)) == ([], 1)
    assert scan("kern:\n\ts_mov_b32 m0, s5\n" + load + "\ts_endpgm\n")[0]
    plain = "kern:\n\tv_cmp_lt_i32_e64 s[4:5], v0, v1\n\tglobal_load_dword v2, v0, s[4:5] offset:16\n\ts_endpgm\n"
    assert scan(plain)[0]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src", SOURCES)
def test_scalar_operands_have_arrived(src, tmp_path):
    out = tmp_path / (src + ".s")
    cmd = [HIPCC, "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "-O3", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    problems, checked = scan(out.read_text())
    print(f"{src}: {checked} loads into LDS checked")
    assert not problems, f"{len(problems)}:\n" + "\n".join(problems[:10])
