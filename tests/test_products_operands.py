"""The generated code of the products whose matrix instructions are written as
assembly, seen from their operands (no GPU needed). A vector instruction's result
may be read by a matrix instruction two wait states later; the compiler inserts
them in front of matrix instructions that it knows, not in front of these. So no
vector instruction of its own may write an operand or a sum right before one. In
the 256 x 256 loops the sums stay where they are: nothing moves one there.

The loads into LDS are assembly, too. A scalar register that a vector instruction
wrote may be read by a load five wait states later (a descriptor that came too late
would send the load anywhere), the LDS address register one wait state after it was
set; and that register is used by the assembly alone."""
import os
import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from combine_get_dispatch_06_amd import build
from test_products_code import MFMA, _kernels, _listing, _registers, _wait_states

NEEDED = 2
NEEDED_SCALAR = 5


def _written(line: str) -> set:
    """Vector registers that a vector instruction writes."""
    if not line.startswith("v_") or line.startswith((MFMA, "v_cmp", "v_readlane", "v_readfirstlane")):
        return set()
    ops = line.split(None, 1)[1].split(",") if " " in line or "\t" in line else []
    return _registers(",".join(ops[:2] if "swap" in line else ops[:1]))


def _scalars(text: str) -> set:
    regs = set()
    for lo, hi, one in re.findall(r"\bs(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        regs |= set(range(int(lo), int(hi) + 1) if lo else [int(one)])
    return regs


def _written_scalars(line: str) -> set:
    """Scalar registers that a vector instruction writes."""
    if not line.startswith(("v_readlane", "v_readfirstlane", "v_cmp")):
        return set()
    return _scalars(line.split(None, 1)[1].split(",")[0])


def late_operands(code, labels):
    """(vector instruction, assembly matrix instruction) pairs that stand too close."""
    return _close(code, labels, NEEDED, _written, lambda line: _registers(line) if line.startswith(MFMA) else set())


def late_descriptors(code, labels):
    """(vector instruction, assembly load) pairs that stand too close."""
    return _close(code, labels, NEEDED_SCALAR, _written_scalars,
                  lambda line: _scalars(line) if line.startswith("buffer_load") else set())


def _close(code, labels, needed, written, read):
    """Pairs of an instruction that writes and one of assembly that reads the same register too soon."""
    found = []
    for start, (ins, _) in enumerate(code):
        result = written(ins)
        if not result:
            continue
        todo, seen = [(start + 1, 0)], set()
        while todo:
            at, passed = todo.pop()
            while at < len(code) and passed < needed and (at, passed) not in seen:
                seen.add((at, passed))
                line, own = code[at]
                if own and read(line) & result:
                    found.append((ins, line))
                    break
                passed += _wait_states(line)
                to = re.match(r"s_c?branch\w*\s+(\.LBB\w+)", line)
                if to:
                    todo.append((labels[to.group(1)], passed))
                if line.startswith(("s_branch", "s_endpgm", "s_setpc")):
                    break
                at += 1
    return found


def main_loop(code, labels):
    """The instructions of the innermost loop around the assembly matrix instructions."""
    own = [i for i, (line, o) in enumerate(code) if o and line.startswith(MFMA)]
    loops = []
    for i, (line, _) in enumerate(code):
        to = re.match(r"s_c?branch\w*\s+(\.LBB\w+)", line)
        if to and labels[to.group(1)] <= own[len(own) // 2] <= i:
            loops.append((i - labels[to.group(1)], labels[to.group(1)], i))
    _, a, z = min(loops)
    return [line for line, _ in code[a:z + 1]]


@pytest.fixture(scope="module")
def every(tmp_path_factory):
    """name -> (code, labels) of all products."""
    files = ["cgd_gemm.hip", "cgd_gemm_fp8.hip", "cgd_gemm_grad.hip"]
    at = tmp_path_factory.mktemp("listings")
    with ThreadPoolExecutor(3) as pool:
        texts = list(pool.map(lambda f: _listing(os.path.join(build.CSRC, f), str(at / (f + ".s"))), files))
    return {name: (code, labels) for text in texts for name, code, labels in _kernels(text)}


@pytest.fixture(scope="module")
def kernels(every):
    """Those with matrix instructions as assembly."""
    return {n: k for n, k in every.items() if any(own and ins.startswith(MFMA) for ins, own in k[0])}


def test_operands_are_there(kernels):
    assert len(kernels) == 4  # forward, FP8 on tall tiles, both gradients
    for name, (code, labels) in kernels.items():
        bad = late_operands(code, labels)
        assert not bad, (name, bad)


def test_sums_stay_in_the_main_loop(kernels):
    tall = {n: k for n, k in kernels.items() if any(o and re.match(r"v_mfma\w* a\[", line) for line, o in k[0])}
    assert len(tall) == 3
    for name, (code, labels) in tall.items():
        loop = main_loop(code, labels)
        assert sum(line.startswith(MFMA) for line in loop) == 128, name  # two halves of a stage
        moved = [line for line in loop if "accvgpr" in line]
        assert not moved, (name, moved)


def test_loads_have_their_descriptors(every):
    assert len(every) == 11
    for name, (code, labels) in every.items():
        assert sum(own and line.startswith("buffer_load") for line, own in code) > 8, name
        bad = late_descriptors(code, labels)
        assert not bad, (name, bad)


def test_the_loads_address_register(every):
    for name, (code, _) in every.items():
        bad = [line for line, own in code if not own and re.search(r"\bm0\b", line)]
        assert not bad, (name, bad)
        for (line, _), (after, _) in zip(code, code[1:]):
            assert not (re.match(r"s_\w+ m0,", line) and after.startswith("buffer_load")), (name, line, after)


@pytest.mark.parametrize("between,late", [([], True), (["s_nop 0"], True), (["s_nop 1"], False),
                                          (["s_add_u32 s0, s0, 1"], True), (["s_add_u32 s0, s0, 1"] * 2, False),
                                          (["v_mfma_x v[8:11], v[40:47], v[48:55], 0"], False)])
@pytest.mark.parametrize("write", ["v_mov_b32_e32 v21, v60", "v_accvgpr_write_b32 a2, v60", "v_permlane16_swap_b32 v60, v21"])
def test_the_check_itself(write, between, late):
    code = [(write, False)] + [(b, True) for b in between] + [("v_mfma_x a[0:3], v[20:27], v[28:35], a[0:3]", True)]
    assert bool(late_operands(code, {})) == late
    code = [("s_branch .LBB1", False), ("s_nop 7", False), (write, False)] + [(b, True) for b in between] + [("s_branch .LBB2", False)]
    code += [("v_mfma_x a[0:3], v[20:27], v[28:35], a[0:3]", True)]
    spent = sum(_wait_states(b) for b in between) + 1  # across a branch, which is a wait state itself
    assert bool(late_operands(code, {".LBB1": 2, ".LBB2": len(code) - 1})) == (spent < NEEDED)


@pytest.mark.parametrize("between,late", [(0, True), (4, True), (5, False)])
@pytest.mark.parametrize("write", ["v_readlane_b32 s6, v184, 62", "v_readfirstlane_b32 s5, v2"])
def test_the_check_of_descriptors_itself(write, between, late):
    code = [(write, False)] + [("s_add_u32 s90, s90, 1", False)] * between + [("buffer_load_dwordx4 v3, s[4:7], 0 offen lds", True)]
    assert bool(late_descriptors(code, {})) == late
