"""The generated code of the products whose matrix instructions are written as
assembly (no GPU needed). The compiler does not know when the results of such
an instruction are there, so nothing may touch them before 20 wait states have
passed (the longest matrix instruction needs 19): a compiler that moved a sum in
between would take it too early. Every instruction is one wait state at least,
s_nop N is N + 1, a matrix instruction 4 at least."""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from combine_get_dispatch_06_amd import build

MFMA = "v_mfma_"
NEEDED = 20


def _wait_states(line: str) -> int:
    nop = re.match(r"s_nop (\d+)", line)
    return int(nop.group(1)) + 1 if nop else 4 if line.startswith(MFMA) else 1


def _listing(src: str, out: str) -> str:
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    r = subprocess.run([os.environ.get("HIPCC", "/opt/rocm/bin/hipcc"), *flags, f"-I{build.INCLUDE}", f"-I{build.CSRC}", "--cuda-device-only", "-S", src, "-o", out],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    return open(out).read()


def _kernels(text: str):
    """-> (name, instructions with their asm flag, label -> index) of each kernel."""
    for m in re.finditer(r"^(_ZN3cgd11gemm_kernel\w+):[^\n]*\n(.*?)^\.Lfunc_end", text, re.M | re.S):
        code, labels, own = [], {}, False
        for line in m.group(2).split("\n"):
            line = line.strip()
            if "#ASMSTART" in line or "#ASMEND" in line:
                own = "#ASMSTART" in line
            elif re.match(r"\.LBB\w+:", line):
                labels[line.split(":")[0]] = len(code)
            elif line and not line.startswith((";", ".", "//")):
                code.append((line.split(";")[0].strip(), own))
        yield m.group(1), code, labels


def _registers(text: str) -> set:
    regs = set()
    for kind, lo, hi, one in re.findall(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        regs |= {kind + str(n) for n in (range(int(lo), int(hi) + 1) if lo else [int(one)])}
    return regs


def early_uses(code, labels):
    """Instructions that touch a result of an assembly matrix instruction too early."""
    found = []
    for start, (ins, own) in enumerate(code):
        if not (own and ins.startswith(MFMA)):
            continue
        result = _registers(ins.split(",")[0])
        todo, seen = [(start + 1, 0)], set()
        while todo:
            at, passed = todo.pop()
            while at < len(code) and (at, passed) not in seen:
                seen.add((at, passed))
                line = code[at][0]
                if passed >= NEEDED:
                    break
                passed += _wait_states(line)
                if not line.startswith(MFMA) and _registers(line.split(None, 1)[1] if " " in line or "\t" in line else "") & result:
                    found.append((ins, line))
                    break
                to = re.match(r"s_c?branch\w*\s+(\.LBB\w+)", line)
                if to:
                    todo.append((labels[to.group(1)], passed))
                if line.startswith(("s_branch", "s_endpgm", "s_setpc")):
                    break
                at += 1
    return found


def test_results_are_not_touched_early(tmp_path):
    files = ["cgd_gemm.hip", "cgd_gemm_fp8.hip", "cgd_gemm_grad.hip"]
    with ThreadPoolExecutor(3) as pool:
        texts = list(pool.map(lambda f: _listing(os.path.join(build.CSRC, f), str(tmp_path / (f + ".s"))), files))
    checked = 0
    for text in texts:
        for name, code, labels in _kernels(text):
            if any(own and ins.startswith(MFMA) for ins, own in code):
                checked += 1
                bad = early_uses(code, labels)
                assert not bad, (name, bad)
    assert checked == 4  # forward, FP8 on tall tiles, both gradients


OTHER = "v_mfma_x v[8:11], v[40:47], v[48:55], 0"


@pytest.mark.parametrize("between,early", [([], True), ([OTHER] * 4, True), ([OTHER] * 5, False), (["s_nop 15"], True),
                                           (["s_nop 15", "s_nop 15"], False), (["s_nop 15"] + ["s_add_u32 s0, s0, 1"] * 4, False)])
def test_the_check_itself(between, early):
    code = [("v_mfma_x v[0:3], v[20:27], v[28:35], 0", True)] + [(b, True) for b in between] + [("v_mov_b32_e32 v60, v2", False)]
    assert bool(early_uses(code, {})) == early
