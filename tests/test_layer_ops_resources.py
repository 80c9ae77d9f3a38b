"""Build guard on the gfx950 code of the operators next to dispatch and
combine: no spills to memory, no packed fp32, the product's operands loaded
straight into LDS and multiplied by the scaled fp4 instruction -- and, as that
instruction stands in inline assembly there, no vector instruction that writes
one of its operands right before it and no read of its sums right behind it,
for which the compiler would otherwise have put wait states."""
import re

import pytest

from test_kernel_resources import _compile

SOURCES = ["route.hip", "mx.hip", "group.hip", "product.hip"]
WAIT_STATES = 3  # a matrix instruction's operands are left alone for these many instructions before it


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    d = str(tmp_path_factory.mktemp("isa"))
    return {src: _compile(src, d) for src in SOURCES}


def test_no_scratch_and_no_spills(compiled):
    for src, (res, _) in compiled.items():
        assert res, f"{src}: no resource remarks parsed"
        for name, r in res.items():
            assert r.get("ScratchSize", 0) == 0, (src, name, r)
            assert r.get("VGPRs Spill", 0) == 0, (src, name, r)


def test_no_packed_fp32_instructions(compiled):
    for src, (_, asm) in compiled.items():
        assert not re.search(r"\bv_pk_(fma|mul|add)_f32\b", asm), src


def test_the_product_uses_the_matrix_cores_and_direct_loads(compiled):
    asm = compiled["product.hip"][1]
    assert re.search(r"v_mfma_scale_f32_16x16x128_f8f6f4 a\[", asm)
    assert re.search(r"buffer_load_dwordx4 .* lds", asm)
    assert re.search(r"v_cvt_scalef32_pk_fp4_bf16", compiled["mx.hip"][1])


def _registers(text):
    m = re.match(r"([va])\[(\d+):(\d+)\]$", text)
    if m:
        return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.match(r"([va])(\d+)$", text)
    return {(m[1], int(m[2]))} if m else set()


def _instructions(asm):
    """(opcode, operands, whether it stands in inline assembly) in order; None at a label."""
    inline = False
    for line in asm.splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            inline = "#ASMSTART" in line
        line = line.split(";")[0].strip()
        if re.match(r"\.?\w+:$", line):
            yield None
        elif line and not line.startswith("."):
            op, _, rest = line.replace("\t", " ").partition(" ")
            yield op, [a.strip().split(" ")[0] for a in rest.split(",")], inline


def test_matrix_instructions_keep_their_distance(compiled):
    asm = compiled["product.hip"][1]
    seen, recent, behind = 0, [], None
    for ins in _instructions(asm):
        if ins is None:
            recent, behind = [], None  # a jump lies between: the loops' ends hold other instructions
            continue
        op, args, inline = ins
        states = int(args[0]) + 1 if op == "s_nop" else 1
        if op.startswith("v_mfma_scale") and inline:
            seen += 1
            operands = set().union(*(_registers(a) for a in args[1:6]))
            passed = 0
            for wrote, n, vector in reversed(recent):
                if passed >= WAIT_STATES:
                    break
                assert not (vector and wrote & operands), (args, wrote)
                passed += n
            behind = (_registers(args[0]), 0) if args[0].startswith("a") else None
        elif behind is not None:
            sums, passed = behind
            if op.startswith("v_accvgpr_read"):
                assert passed >= 8 or not (_registers(args[1]) & sums), (op, args)
            behind = (sums, passed + states)
        recent.append((_registers(args[0]) if args else set(), states, op.startswith("v_") and not op.startswith("v_mfma")))
        del recent[:-8]
    assert seen > 1000
