"""Every kernel of the experts' products in bf16 and int8, at every number of
steps of the summed index and each of its endings: the 256 x 256 tiles need
shapes that test_gpu_expert_ops.py does not have.  test_expert_ops_plans.py
holds that these shapes reach the kernels named here."""
import pytest
import torch

import combine_count_amd as epdc
import expert_oracle as O

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
KIND = {BF16: epdc.EPDC_BF16, FP32: epdc.EPDC_FP32}
SIZES = [700, 0, 1, 256, 515]  # entries of the experts
LONG = 21896                   # columns (of the product; of the rows' gradient): 86 tiles of 256, the last a part
SHORT = 1160                   # columns of the product for tiles of 128: 10 of them, the last a part
# elements of the summed index: 1 to 5 steps of 128 bytes, whole and with endings
BF16_TERMS = [8, 56, 64, 72, 120, 128, 136, 192, 200, 256, 264, 320]
INT8_TERMS = [16, 112, 128, 144, 256, 272, 384, 400, 512, 528]
# the weights' gradient: entries of the experts (steps of 64)
GRAD_SIZES = [0, 1, 63, 64, 65, 128, 129, 193, 700]
GRAD_SHAPE = (1288, 1544)      # 6 x 7 tiles of 256 an expert


def product_shapes():
    """(form, kind, experts, columns, hidden, maxEntries), kinds 0: product, 1: rows' gradient, 2: weights' gradient"""
    n = sum(SIZES)
    out = [(form, 0, len(SIZES), cols, t, n) for form, cols in (("tiles256", LONG), ("tiles128", SHORT)) for t in BF16_TERMS + INT8_TERMS]
    out += [("tiles256", 1, len(SIZES), t, LONG, n) for t in BF16_TERMS]
    return out + [("tiles256", 2, len(GRAD_SIZES), *GRAD_SHAPE, sum(GRAD_SIZES))]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _offsets(sizes):
    o = [0]
    for s in sizes:
        o.append(o[-1] + s)
    return o, torch.tensor(o, dtype=torch.int32, device="cuda")


def _check(got, ref, bound, what):
    got = got.double()
    bad = ~((got - ref).abs() <= bound) & ~(got == ref)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist())


def _rows(g, n, R):
    row = torch.randint(R, (n,), device="cuda", generator=g, dtype=torch.int32)
    row[::97] = -1
    row[5::101] = R
    return row


@pytest.mark.parametrize("cols", [LONG, SHORT], ids=["tiles256", "tiles128"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("terms", BF16_TERMS)
def test_product_tiles(terms, dtype, cols):
    g = _gen(terms)
    o, off = _offsets(SIZES)
    n, R = o[-1], 901
    x = torch.randn(R, terms, device="cuda", generator=g).to(BF16)
    b = torch.randn(len(SIZES), cols, terms, device="cuda", generator=g).to(BF16)
    row, w = _rows(g, n, R), torch.randn(n, device="cuda", generator=g)
    out = torch.full((n + 2, cols), 5.0, device="cuda", dtype=dtype)
    epdc.epdc_expert_linear(len(SIZES), cols, terms, n, R, x, off, row, w, b, out, KIND[dtype])
    ref, size = O.product(x, o, row, w, b, n, out)
    _check(out, ref, O.product_bound(ref, size, terms, dtype), terms)
    assert (out[n:] == 5).all()


@pytest.mark.parametrize("cols", [LONG, SHORT], ids=["tiles256", "tiles128"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("terms", INT8_TERMS)
def test_product_int8_tiles(terms, dtype, cols):
    g = _gen(terms)
    o, off = _offsets(SIZES)
    n, R = o[-1], 901
    x = torch.randint(-127, 128, (R, terms), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
    b = torch.randint(-127, 128, (len(SIZES), cols, terms), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
    sx, sb = torch.rand(R, device="cuda", generator=g), torch.rand(len(SIZES), cols, device="cuda", generator=g)
    row, w = _rows(g, n, R), torch.randn(n, device="cuda", generator=g)
    out = torch.full((n + 2, cols), 5.0, device="cuda", dtype=dtype)
    epdc.epdc_expert_linear_int(len(SIZES), cols, terms, n, R, x, sx, off, row, w, b, sb, out, KIND[dtype])
    ref, _ = O.product(x, o, row, w, b, n, out, sx, sb)
    _check(out, ref, O.int8_bound(ref, dtype), terms)
    assert (out[n:] == 5).all()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("terms", BF16_TERMS)
def test_rows_grad_tiles256(terms, dtype):
    g = _gen(terms)
    o, off = _offsets(SIZES)
    n, R = o[-1], 901
    d = torch.randn(R, terms, device="cuda", generator=g).to(BF16)
    b = torch.randn(len(SIZES), terms, LONG, device="cuda", generator=g).to(BF16)
    row, w = _rows(g, n, R), torch.randn(n, device="cuda", generator=g)
    out = torch.full((n + 2, LONG), 5.0, device="cuda", dtype=dtype)
    epdc.epdc_expert_rows_grad(len(SIZES), terms, LONG, n, R, d, off, row, w, b, out, KIND[dtype])
    ref, size = O.product(d, o, row, w, b, n, out, transposed=True)
    _check(out, ref, O.product_bound(ref, size, terms, dtype), terms)
    assert (out[n:] == 5).all()


@pytest.mark.parametrize("gather", [False, True], ids=["in_order", "gathered"])
@pytest.mark.parametrize("base", [False, True], ids=["alone", "added"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_weights_grad_tiles256(dtype, base, gather):
    g = _gen(11)
    N, H = GRAD_SHAPE
    o, off = _offsets(GRAD_SIZES)
    n, E = o[-1], len(GRAD_SIZES)
    R = 555 if gather else n
    x = torch.randn(R, H, device="cuda", generator=g).to(BF16)
    d = torch.randn(n, N, device="cuda", generator=g).to(BF16)
    row = _rows(g, n, R) if gather else None
    out_row = torch.randperm(n, device="cuda", generator=g).to(torch.int32) if gather else None
    b = torch.randn(E, N, H, device="cuda", generator=g).to(dtype) if base else None
    out = torch.full((E, N, H), 5.0, device="cuda", dtype=dtype)
    epdc.epdc_expert_weights_grad(E, N, H, n, n, d, out_row, R, x, row, off, b, out, KIND[dtype])
    ref, size = O.weights_grad(d, out_row, x, row, o, n, E, b)
    _check(out, ref, O.product_bound(ref, size, max(GRAD_SIZES), dtype), "weights")


def test_tiles256_special_values_and_repeats():
    """A NaN row and infinities next to the end of the summed index stay where they belong, the result is the same
    from run to run."""
    g = _gen(5)
    o, off = _offsets(SIZES)
    n, terms = o[-1], 72
    x = torch.randn(n, terms, device="cuda", generator=g).to(BF16)
    x[3], x[9, terms - 1], x[700, 0] = float("nan"), float("inf"), float("inf")
    b = torch.randn(len(SIZES), LONG, terms, device="cuda", generator=g).to(BF16)
    b[0, 5, terms - 1], b[3, LONG - 1] = float("inf"), float("nan")
    b[0, 7] = 0.0
    outs = []
    for _ in range(2):
        out = torch.full((n, LONG), 5.0, device="cuda")
        epdc.epdc_expert_linear(len(SIZES), LONG, terms, n, n, x, off, None, None, b, out, epdc.EPDC_FP32)
        outs.append(out)
    ref, size = O.product(x, o, None, None, b, n, outs[0])
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(outs[0]), torch.isnan(ref)) and torch.equal(torch.isfinite(outs[0]), fine)
    _check(outs[0][fine], ref[fine], O.product_bound(ref, size, terms, FP32)[fine], "product")
    assert torch.equal(outs[0].view(torch.int32), outs[1].view(torch.int32))
