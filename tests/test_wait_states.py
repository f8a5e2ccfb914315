"""The hand-placed matrix instructions keep their distances in the code the compiler makes of them.

The large products write their matrix instructions as asm, around which the compiler places no wait states. What the
hardware needs is, between a vector instruction that writes one of their operands and the matrix instruction, two wait
states; and between the matrix instruction and any other access to its result, 19 (a following one may add to the same
result). This reads the assembly of the kernels' file, built with the library's flags, and counts them: an instruction
is one wait state, `s_nop n` n + 1.
"""
import os
import re
import shutil
import subprocess

import pytest

from moe_expert_load_ultraep_amd import _build

BEFORE, BEHIND = 2, 19
REG = re.compile(r"\b([av])(?:\[(\d+):(\d+)\]|(\d+))")


def registers(text):
    found = set()
    for kind, lo, hi, one in REG.findall(text):
        found |= {(kind, r) for r in (range(int(lo), int(hi) + 1) if lo else [int(one)])}
    return found


def violations(lines):
    """Distances that one function's assembly lines do not keep; and how many matrix instructions in asm it has."""
    bad, count, in_asm = [], 0, False
    written, results = [], {}      # [(state, registers)] of the last vector instructions; register: state of its product
    state = 0
    for line in lines:
        if "#ASMSTART" in line or "#ASMEND" in line:
            in_asm = "#ASMSTART" in line
            continue
        code = line.split(";")[0].split("//")[0].strip()
        if not code or code.startswith(".") and not code.endswith(":"):
            continue
        late = [r for r, at in results.items() if state - at < BEHIND + 1]
        if code.endswith(":") or code.startswith(("s_cbranch", "s_branch", "s_endpgm", "s_setpc")):
            if late:
                bad.append(f"{code}: results under way where paths meet or part")
                results = {}
            state += not code.endswith(":")
            continue
        op, _, rest = code.partition(" ")
        if op == "s_nop":
            state += int(rest) + 1
            continue
        operands = [p.strip() for p in rest.split(",")]
        if op.startswith("v_mfma") and in_asm:
            count += 1
            d, a, b, c = (registers(p) for p in operands[:4])
            for at, regs in written:
                if state - at < BEFORE + 1 and regs & (a | b | c):
                    bad.append(f"{code}: operand written {state - at - 1} wait states before")
            if (a | b) & set(late):
                bad.append(f"{code}: multiplies a result under way")
            if c & set(late) and c != d:
                bad.append(f"{code}: adds to a result under way elsewhere")
            results.update({r: state for r in d})
        else:
            if registers(rest) & set(late):
                bad.append(f"{code}: touches a result under way")
            if op.startswith("v_") and not op.startswith(("v_mfma", "v_cmp")):
                regs = registers(operands[0]) | (registers(operands[1]) if op.startswith("v_swap") else set())
                written = [w for w in written if state - w[0] < BEFORE + 1] + [(state, regs)]
        state += 1
    return bad, count


def functions(text):
    """{name: lines} of the assembly's functions."""
    found, name = {}, None
    for line in text.splitlines():
        m = re.match(r"(_Z\w+):", line)
        if m:
            name = m.group(1)
            found[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name:
            found[name].append(line)
    return found


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs hipcc")
def test_products_keep_their_distances(tmp_path):
    out = str(tmp_path / "gemm.s")
    cmd = [a for a in _build.command(out) if a not in ("-shared", "-fPIC") and not a.endswith(".hip")]
    cmd += ["--cuda-device-only", "-S", os.path.join(_build.CSRC, "ultraep_gemm.hip")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    counts = {}
    for name, lines in functions(open(out).read()).items():
        bad, counts[name] = violations(lines)
        assert not bad, (name, bad[:5], len(bad))
    # two blocks of 32 steps by 8 fragments of B, and by 4
    assert [n for n in counts.values() if n] == [2 * 32 * 8 + 2 * 32 * 4] * 2, counts


MFMA = ["\t;;#ASMSTART", "\tv_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]", "\t;;#ASMEND"]


@pytest.mark.parametrize("lines,ok", [
    (["\tv_mov_b32_e32 v5, 0", "\ts_nop 1"] + MFMA, True),
    (["\tv_mov_b32_e32 v5, 0", "\ts_nop 0"] + MFMA, False),
    (["\tv_mov_b32_e32 v5, 0", "\tv_mov_b32_e32 v9, 0"] + MFMA, False),
    (["\tv_accvgpr_write_b32 a3, 0"] + MFMA, False),
    (["\tv_mov_b32_e32 v8, 0"] + MFMA + MFMA, True),
    (MFMA + ["\ts_nop 15", "\ts_nop 2", "\tv_accvgpr_read_b32 v1, a0"], True),
    (MFMA + ["\ts_nop 15", "\ts_nop 1", "\tv_accvgpr_read_b32 v1, a0"], False),
    (MFMA + ["\tglobal_store_dwordx4 v[0:1], a[0:3], off"], False),
    (MFMA + ["\ts_nop 15", "\ts_cbranch_vccnz .LBB0_1"], False),
    (MFMA + ["\ts_nop 15", "\ts_nop 3", ".LBB0_1:", "\tv_accvgpr_read_b32 v1, a0"], True),
    (MFMA + [".LBB0_1:"], False),
])
def test_counting(lines, ok):
    bad, count = violations(lines)
    assert (not bad) == ok and count >= 1
