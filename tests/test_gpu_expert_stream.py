"""The products of one to four experts with few entries (weights streamed into
registers), with many 128-byte chunks of a row for each of a block's four
waves: every remainder of the chunks after the steady loop, rows that end inside
a chunk, in bf16 and int8.  Whole numbers, whose sums are exact, and weights and
scales that are powers of two: results are equal to the formula's, rounded once.
test_expert_ops_plans.py holds that these shapes reach the kernels named here."""
import pytest
import torch

import combine_count_amd as epdc
import expert_oracle as O

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
KIND = {BF16: epdc.EPDC_BF16, FP32: epdc.EPDC_FP32}
COLS = 200  # of 32 a block, the last a part
# entries of the experts
GROUPS = {
    "stream16": [[1], [16], [3, 14], [0, 20, 1, 12]],
    "stream64": [[17], [64], [256], [65, 85], [140, 0, 3, 157]],
}
# whole chunks of a row: twelve in a row are every remainder of three and of two rounds of four waves
BF16_CHUNKS = list(range(24, 36)) + [112]
INT8_CHUNKS = list(range(25, 37)) + [56]
BF16_ENDS = [0, 8, 40, 56]    # elements behind the last whole chunk of 64
INT8_ENDS = [0, 16, 64, 112]  # of 128


def shapes():
    """(form, kind, experts, columns, hidden, maxEntries) of every case"""
    out = []
    for form, groups in GROUPS.items():
        for sizes in groups:
            for chunk, chunks, ends in ((64, BF16_CHUNKS, BF16_ENDS), (128, INT8_CHUNKS, INT8_ENDS)):
                out += [(form, 0, len(sizes), COLS, c * chunk + end, sum(sizes)) for c in chunks for end in ends]
    return out


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _powers(g, *shape):
    return torch.exp2(torch.randint(-2, 3, shape, device="cuda", generator=g).float())


def _entries(sizes, g, R):
    o = [0]
    for s in sizes:
        o.append(o[-1] + s)
    row = torch.randint(R, (o[-1],), device="cuda", generator=g, dtype=torch.int32)
    row[9::23] = -1
    row[11::29] = R
    return o, torch.tensor(o, dtype=torch.int32, device="cuda"), row


@pytest.mark.parametrize("chunks", BF16_CHUNKS)
@pytest.mark.parametrize("form", list(GROUPS))
def test_streamed_product(form, chunks):
    g = _gen(chunks)
    for end in BF16_ENDS:
        H, R = 64 * chunks + end, 40
        # products of at most 16, sums below 16 * 7224 < 2^24
        x = torch.randint(-4, 5, (R, H), device="cuda", generator=g).to(BF16)
        b = torch.randint(-4, 5, (4, COLS, H), device="cuda", generator=g).to(BF16)
        for sizes in GROUPS[form]:
            o, off, row = _entries(sizes, g, R)
            n, w = o[-1], _powers(g, o[-1])
            for dtype in (BF16, FP32):
                out = torch.full((n + 1, COLS), 5.0, device="cuda", dtype=dtype)
                epdc.epdc_expert_linear(len(sizes), COLS, H, n, R, x, off, row, w, b, out, KIND[dtype])
                ref, _ = O.product(x, o, row, w, b, n, out)
                assert torch.equal(out, ref.to(dtype)), (H, sizes, dtype)


@pytest.mark.parametrize("chunks", INT8_CHUNKS)
@pytest.mark.parametrize("form", list(GROUPS))
def test_streamed_product_int8(form, chunks):
    g = _gen(chunks)
    for end in INT8_ENDS:
        H, R = 128 * chunks + end, 40
        x = torch.randint(-128, 128, (R, H), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
        b = torch.randint(-128, 128, (4, COLS, H), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
        sx, sb = _powers(g, R), _powers(g, 4, COLS)
        for sizes in GROUPS[form]:
            o, off, row = _entries(sizes, g, R)
            n, w = o[-1], _powers(g, o[-1])
            for dtype in (BF16, FP32):
                out = torch.full((n + 1, COLS), 5.0, device="cuda", dtype=dtype)
                epdc.epdc_expert_linear_int(len(sizes), COLS, H, n, R, x, sx, off, row, w, b, sb, out, KIND[dtype])
                ref, _ = O.product(x, o, row, w, b, n, out, sx, sb)
                # the sum as fp32, products with powers of two, the output's rounding
                assert torch.equal(out, ref.float().to(dtype)), (H, sizes, dtype)
