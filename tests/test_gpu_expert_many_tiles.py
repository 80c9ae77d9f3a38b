"""The 128 x 128 tiles of the products and of the rows' gradient where a block
takes several one behind the other (512 blocks run at once on 256 CUs): the next
tile's first steps are requested while the last ones of a tile are computed, and
its results are on their way behind them.  At every number of steps and each of
their endings, tiles of one and of two fragments of rows in turn.  Whole
numbers, whose sums are exact, and weights and scales that are powers of two:
results are equal to the formula's, rounded once.  test_expert_ops_plans.py holds
that these shapes reach that kernel, with tiles for two rounds and a half."""
import pytest
import torch

import combine_count_amd as epdc
import expert_oracle as O

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
KIND = {BF16: epdc.EPDC_BF16, FP32: epdc.EPDC_FP32}
SIZES = [200, 0, 1, 128, 65, 300, 63, 243]  # entries of the experts: 11 tiles of rows
COLS = 16392                                # 129 tiles of columns, the last a part
BLOCKS = 512                                # that run at once
# elements of the summed index: 1 to 6 steps of 128 bytes, whole and with endings
BF16_TERMS = [8, 64, 72, 128, 136, 192, 200, 256, 320, 328]
INT8_TERMS = [16, 128, 144, 256, 272, 384, 512, 528, 640]


def tiles():
    return sum(-(-s // 128) for s in SIZES) * -(-COLS // 128)


def shapes():
    """(form, kind, experts, columns, hidden, maxEntries) of every case, kinds 0: product, 1: rows' gradient"""
    n = sum(SIZES)
    out = [("tiles128", 0, len(SIZES), COLS, t, n) for t in BF16_TERMS + INT8_TERMS]
    return out + [("tiles128", 1, len(SIZES), t, COLS, n) for t in BF16_TERMS]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _powers(g, *shape):
    return torch.exp2(torch.randint(-2, 3, shape, device="cuda", generator=g).float())


def _entries(g, R):
    o = [0]
    for s in SIZES:
        o.append(o[-1] + s)
    row = torch.randint(R, (o[-1],), device="cuda", generator=g, dtype=torch.int32)
    row[::97] = -1
    row[5::101] = R
    return o, torch.tensor(o, dtype=torch.int32, device="cuda"), row


def _small(g, *shape):
    return torch.randint(-4, 5, shape, device="cuda", generator=g, dtype=torch.int8).to(BF16)


@pytest.mark.parametrize("terms", BF16_TERMS)
@pytest.mark.parametrize("rows_grad", [False, True], ids=["product", "rows_grad"])
def test_bf16_tiles_in_a_row(rows_grad, terms):
    g, R, E = _gen(terms), 901, len(SIZES)
    o, off, row = _entries(g, R)
    n, w = o[-1], _powers(g, o[-1])
    x = _small(g, R, terms)
    b = _small(g, *((E, terms, COLS) if rows_grad else (E, COLS, terms)))
    for dtype in (BF16, FP32):
        out = torch.full((n + 2, COLS), 5.0, device="cuda", dtype=dtype)
        if rows_grad:
            epdc.epdc_expert_rows_grad(E, terms, COLS, n, R, x, off, row, w, b, out, KIND[dtype])
        else:
            epdc.epdc_expert_linear(E, COLS, terms, n, R, x, off, row, w, b, out, KIND[dtype])
        ref, _ = O.product(x, o, row, w, b, n, out, transposed=rows_grad)
        assert torch.equal(out, ref.to(dtype)), dtype


@pytest.mark.parametrize("terms", INT8_TERMS)
def test_int8_tiles_in_a_row(terms):
    g, R, E = _gen(terms), 901, len(SIZES)
    o, off, row = _entries(g, R)
    n, w = o[-1], _powers(g, o[-1])
    x = torch.randint(-127, 128, (R, terms), device="cuda", generator=g, dtype=torch.int8)
    b = torch.randint(-127, 128, (E, COLS, terms), device="cuda", generator=g, dtype=torch.int8)
    sx, sb = _powers(g, R), _powers(g, E, COLS)
    for dtype in (BF16, FP32):
        out = torch.full((n + 2, COLS), 5.0, device="cuda", dtype=dtype)
        epdc.epdc_expert_linear_int(E, COLS, terms, n, R, x, sx, off, row, w, b, sb, out, KIND[dtype])
        ref, _ = O.product(x, o, row, w, b, n, out, sx, sb)
        # sums below 127 * 127 * 640 < 2^24: exact in fp32
        assert torch.equal(out, ref.to(dtype)), dtype
