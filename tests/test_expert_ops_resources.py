"""Build guard on the gfx950 code of the experts in bf16 and int8: no spills to
memory, no packed fp32; and of the products' kernels, whose matrix instructions
and loads into LDS stand in inline assembly: nothing but that assembly touches
the accumulation registers that hold the sums, no vector instruction writes an
operand right before a matrix instruction, no sum is read right behind one, and
m0 is set by that assembly only."""
import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_kernel_resources import _compile
from test_layer_ops_resources import _instructions, _registers

PRODUCTS = ["dense_linear.hip", "dense_linear_int.hip", "dense_rows_grad.hip", "dense_weights_grad.hip"]
SOURCES = PRODUCTS + ["gate.hip", "int8.hip"]
WAIT_STATES = 3   # a matrix instruction's operands are left alone for these many instructions before it
READ_STATES = 18  # and its sums, behind it


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    d = str(tmp_path_factory.mktemp("isa"))
    with ThreadPoolExecutor(8) as pool:
        return dict(zip(SOURCES, pool.map(lambda src: _compile(src, d), SOURCES)))


def _kernels(compiled, part="dense_tile_kernel"):
    """(name, code) of the products' kernels whose name holds `part`"""
    name, lines = None, []
    for line in (line for src in PRODUCTS for line in compiled[src][1].splitlines()):
        if line.startswith("_Z") and line.split(";")[0].rstrip().endswith(":"):
            name, lines = line.split(":")[0], []
        elif line.startswith(".Lfunc_end"):
            if name and part in name:
                yield name, "\n".join(lines)
            name = None
        elif name:
            lines.append(line)


def test_no_scratch_and_no_spills(compiled):
    for src, (res, _) in compiled.items():
        kernels = {name: r for name, r in res.items() if "kernel" in name}
        assert kernels, src
        for name, r in kernels.items():
            assert r.get("VGPRs Spill", 0) == 0, (src, name, r)
            if "int8" not in src:  # the 64-bit exponential is called there, on a stack
                assert r.get("ScratchSize", 0) == 0, (src, name, r)


def test_no_packed_fp32_instructions(compiled):
    for src, (_, asm) in compiled.items():
        assert not re.search(r"\bv_pk_(fma|mul|add)_f32\b", asm), src


def test_tiles_keep_two_blocks_per_cu(compiled):
    for src in PRODUCTS:
        for name, r in compiled[src][0].items():
            if "Li128ELi128" in name:
                assert r["Occupancy"] == 2 and r["LDS Size"] <= 80 * 1024, (name, r)


def test_the_sums_registers_are_the_assemblys_own(compiled):
    seen = 0
    for name, body in _kernels(compiled):
        seen += 1
        sums = {("a", i) for i in range(256 if "Li256ELi256" in name else 64)}
        for ins in _instructions(body):
            if ins is None or ins[2]:
                continue
            used = set().union(*(_registers(a) for a in ins[1])) if ins[1] else set()
            assert not used & sums, (name, ins)
    assert seen == 16  # four kinds, two types of output, two tiles


def test_matrix_instructions_keep_their_distance(compiled):
    seen, recent, behind = 0, [], 99
    for ins in (ins for _, body in _kernels(compiled) for ins in _instructions(body)):
        if ins is None:
            recent, behind = [], 99  # a jump lies between: mfma_done stands behind the loops, its wait is 32 states
            continue
        op, args, _ = ins
        states = int(args[0]) + 1 if op == "s_nop" else 1
        if op.startswith("v_mfma"):
            seen += 1
            operands = set().union(*(_registers(a) for a in args[1:3]))
            passed = 0
            for wrote, n, vector in reversed(recent):
                if passed >= WAIT_STATES:
                    break
                assert not (vector and wrote & operands), (args, wrote)
                passed += n
            behind = 0
        else:
            if op.startswith("v_accvgpr_read"):
                assert behind >= READ_STATES, args
            behind += states
        recent.append((_registers(args[0]) if args else set(), states, op.startswith("v_") and not op.startswith("v_mfma")))
        del recent[:-8]
    assert seen > 1000


def test_m0_is_the_assemblys_own(compiled):
    for _, body in _kernels(compiled):
        for ins in _instructions(body):
            if ins is not None and "m0" in ins[1]:
                assert ins[2], ins

