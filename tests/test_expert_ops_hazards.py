"""Build guard on the gfx950 code of the products' kernels (bf16, int8, fp4),
along every path through it, loops' ends and jumps among them: where inline
assembly takes the compiler's place, the wait states that it would have put in.

- No vector instruction writes an operand of a matrix instruction right before it.
- No sum is read right behind a matrix instruction.
- No vector instruction writes a scalar register that a load of the inline
  assembly takes its address from, within the five states that memory
  instructions need.

And of the int8 rows' kernels: only the activation's, which calls a 64-bit
exponential out of line, has a stack."""
import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_kernel_resources import _compile

DENSE = ["dense_linear.hip", "dense_linear_int.hip", "dense_rows_grad.hip", "dense_weights_grad.hip"]
SOURCES = DENSE + ["product.hip", "int8.hip"]
OPERAND_STATES = 3  # between a vector write and the matrix instruction that reads it
READ_STATES = 18    # between a matrix instruction and the read of its sums
SCALAR_STATES = 5   # between a vector write of a scalar register and the load that reads it


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    d = str(tmp_path_factory.mktemp("isa"))
    with ThreadPoolExecutor(8) as pool:
        return dict(zip(SOURCES, pool.map(lambda src: _compile(src, d), SOURCES)))


def registers(text):
    """{(file, number)} of an operand such as v7, a[0:15], s[4:5], vcc"""
    text = text.lstrip("-|").rstrip("|")
    if text in ("vcc", "exec", "m0"):
        return {(text, 0)}
    m = re.match(r"([vas])\[(\d+):(\d+)\]$", text)
    if m:
        return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.match(r"([vas])(\d+)$", text)
    return {(m[1], int(m[2]))} if m else set()


class Code:
    """A kernel's instructions (opcode, operands, whether inline) and, of each, those that may come right before."""

    def __init__(self, text):
        self.ins, before, labels, inline, falls, here = [], [], {}, False, False, []
        for line in text.splitlines():
            if "#ASMSTART" in line or "#ASMEND" in line:
                inline = "#ASMSTART" in line
            line = line.split(";")[0].strip()
            label = re.match(r"([.\w$]+):$", line)
            if label:
                here.append(label[1])
            elif line and not line.startswith("."):
                op, _, rest = line.replace("\t", " ").partition(" ")
                at = len(self.ins)
                for name in here:
                    labels[name] = at
                here = []
                before.append([at - 1] if falls else [])
                self.ins.append((op, [a.strip().split(" ")[0] for a in rest.split(",")], inline))
                falls = op not in ("s_branch", "s_endpgm", "s_setpc_b64")
        for at, (op, args, _) in enumerate(self.ins):
            if op == "s_branch" or op.startswith("s_cbranch"):
                before[labels[args[0]]].append(at)
        self.before = before

    def states(self, at):
        op, args, _ = self.ins[at]
        return int(args[0]) + 1 if op == "s_nop" else 1

    def within(self, at, states):
        """Instructions from which instruction `at` follows with fewer than `states` states between."""
        seen, todo = {}, [(i, 0) for i in self.before[at]]
        while todo:
            i, passed = todo.pop()
            if passed >= states or seen.get(i, states) <= passed:
                continue
            seen[i] = passed
            todo += [(j, passed + self.states(i)) for j in self.before[i]]
        return seen

    def written_by_vector(self, at):
        op, args, _ = self.ins[at]
        if not op.startswith("v_") or op.startswith("v_mfma"):
            return set()
        out = registers(args[0])
        if "_co_" in op or "div_scale" in op or "swap" in op:
            out |= registers(args[1])
        return out


def operands_written(code):
    """(instructions looked at, [(matrix instruction, write)]): writes of its operands right before"""
    seen, bad = 0, []
    for at, (op, args, inline) in enumerate(code.ins):
        if op.startswith("v_mfma") and inline:
            seen += 1
            reads = set().union(*(registers(a) for a in args[1:] if not a.startswith("a")))
            bad += [(args, code.ins[i]) for i in code.within(at, OPERAND_STATES) if code.written_by_vector(i) & reads]
    return seen, bad


def sums_read(code):
    seen, bad = 0, []
    for at, (op, args, inline) in enumerate(code.ins):
        if op.startswith("v_accvgpr_read") and inline:
            seen += 1
            bad += [(args, code.ins[i]) for i in code.within(at, READ_STATES) if code.ins[i][0].startswith("v_mfma")]
    return seen, bad


def addresses_written(code):
    seen, bad = 0, []
    for at, (op, args, inline) in enumerate(code.ins):
        reads = {r for a in args for r in registers(a) if r[0] == "s"}
        if inline and re.match(r"(global|buffer|flat|scratch)_", op) and reads:
            seen += 1
            bad += [(op, args, code.ins[i]) for i in code.within(at, SCALAR_STATES) if code.written_by_vector(i) & reads]
    return seen, bad


def kernels(compiled, sources, part):
    for src in sources:
        name, lines = None, []
        for line in compiled[src][1].splitlines():
            if line.startswith("_Z") and line.split(";")[0].rstrip().endswith(":"):
                name, lines = line.split(":")[0], []
            elif line.startswith(".Lfunc_end"):
                if name and part in name:
                    yield name, Code("\n".join(lines))
                name = None
            elif name:
                lines.append(line)


@pytest.mark.parametrize("check,text,count", [
    # the write lies at the loop's end, the matrix instruction at its head
    (operands_written, "v_mov_b32 v9, v1\n.L0:\n;#ASMSTART\nv_mfma_f32_32x32x16_bf16 a[0:15], v[4:7], v[8:11], 0\n;#ASMEND\n"
                       "s_nop 7\nv_mov_b32 v5, v2\ns_cbranch_scc1 .L0\ns_endpgm", 2),
    (operands_written, ".L0:\n;#ASMSTART\nv_mfma_f32_32x32x16_bf16 a[0:15], v[4:7], v[8:11], 0\n;#ASMEND\n"
                       "v_mov_b32 v5, v2\ns_nop 1\ns_cbranch_scc1 .L0\ns_endpgm", 0),
    # past a jump only
    (operands_written, "v_permlane32_swap_b32 v1, v8\ns_branch .L1\nv_mov_b32 v4, v1\n.L1:\n;#ASMSTART\n"
                       "v_mfma_f32_32x32x16_bf16 a[0:15], v[4:7], v[8:11], 0\n;#ASMEND\ns_endpgm", 2),
    (sums_read, ";#ASMSTART\nv_mfma_f32_32x32x16_bf16 a[0:15], v[4:7], v[8:11], 0\n;#ASMEND\ns_nop 15\n.L2:\n;#ASMSTART\n"
                "v_accvgpr_read_b32 v1, a0\n;#ASMEND\ns_endpgm", 1),
    (sums_read, ";#ASMSTART\nv_mfma_f32_32x32x16_bf16 a[0:15], v[4:7], v[8:11], 0\n;#ASMEND\ns_nop 15\ns_nop 15\n.L2:\n"
                ";#ASMSTART\nv_accvgpr_read_b32 v1, a0\n;#ASMEND\ns_endpgm", 0),
    (addresses_written, "v_readfirstlane_b32 s4, v1\n;#ASMSTART\ns_add_u32 m0, s9, 0\ns_nop 0\n"
                        "global_load_lds_dwordx4 v3, s[4:5]\n;#ASMEND\ns_endpgm", 1),
    (addresses_written, "v_readfirstlane_b32 s4, v1\ns_nop 2\n;#ASMSTART\ns_add_u32 m0, s9, 0\ns_nop 0\n"
                        "global_load_lds_dwordx4 v3, s[4:5]\n;#ASMEND\ns_endpgm", 0),
    (addresses_written, ".L3:\n;#ASMSTART\nglobal_load_lds_dwordx4 v3, s[4:5]\n;#ASMEND\nv_cmp_eq_u32_e64 s[4:5], v1, v2\n"
                        "s_cbranch_vccnz .L3\ns_endpgm", 1),
])
def test_the_checks_find_what_they_look_for(check, text, count):
    seen, bad = check(Code(text))
    assert seen == 1 and len(bad) == count, bad


def test_matrix_instructions_operands_are_settled(compiled):
    for sources, part, least in ((DENSE, "dense_tile_kernel", 1000), (["product.hip"], "", 1000)):
        total = 0
        for name, code in kernels(compiled, sources, part):
            seen, bad = operands_written(code)
            total += seen
            assert not bad, (name, bad[:3])
        assert total > least, sources


def test_sums_are_read_behind_the_matrix_instructions(compiled):
    total = 0
    for name, code in kernels(compiled, DENSE, "dense_tile_kernel"):
        seen, bad = sums_read(code)
        total += seen
        assert not bad, (name, bad[:3])
    assert total > 1000


def test_loads_addresses_are_settled(compiled):
    total = 0
    for name, code in kernels(compiled, DENSE, "dense_tile_kernel"):
        seen, bad = addresses_written(code)
        total += seen
        assert not bad, (name, bad[:3])
    assert total > 50


def test_only_the_activation_in_codes_has_a_stack(compiled):
    res = {name: r for name, r in compiled["int8.hip"][0].items() if "kernel" in name}
    plain = {name: r for name, r in res.items() if "gate_int_kernel" not in name}
    assert len(plain) == 4 and len(res) == 8
    for name, r in plain.items():
        assert r.get("ScratchSize", 0) == 0 and r.get("VGPRs Spill", 0) == 0, (name, r)
