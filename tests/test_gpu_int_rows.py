"""Scales and codes of int8 rows follow the definition to the last bit whatever
the row's largest magnitude is: the scale is the fp32 quotient by 127, not a
product with a rounded 1 / 127 (which is a step off for some significands, and
sends exact ties to other codes)."""
import pytest
import torch

import combine_count_amd as epdc
import expert_oracle as O

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
KIND = {BF16: epdc.EPDC_BF16, FP32: epdc.EPDC_FP32}


def _rows(dtype, cols):
    """A row for every significand of bf16 (fp32: and its neighbours), at seven exponents, and its values: the
    largest, halves of codes of it as near as the type has them, then random ones."""
    significand = 1.0 + torch.arange(128, dtype=torch.float64) / 128
    if dtype == FP32:
        significand = torch.cat([significand, significand + 2.0 ** -23, 2.0 - 2.0 ** -23 * torch.arange(1, 9, dtype=torch.float64)])
    most = (significand[:, None] * 2.0 ** torch.tensor([-120.0, -40, -8, 0, 1, 30, 110], dtype=torch.float64)).flatten()
    x = most[:, None] * (2 * torch.rand(len(most), cols, dtype=torch.float64, generator=torch.Generator().manual_seed(cols)) - 1)
    ties = (torch.arange(127, dtype=torch.float64) + 0.5) / 127
    x[:, :127] = most[:, None] * ties
    x[:, 127] = -most
    return x.to(dtype).cuda()


@pytest.mark.parametrize("cols", [128, 1040])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_every_significand(dtype, cols):
    x = _rows(dtype, cols)
    q, s = torch.zeros(x.shape, dtype=torch.int8, device="cuda"), torch.zeros(len(x), device="cuda")
    epdc.epdc_int_quantize(1, len(x), cols, KIND[dtype], x, None, q, s)
    rq, rs = O.int8_rows(x)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)
    other = x.float().abs().amax(1).cpu() * torch.tensor(1.0 / 127.0, dtype=torch.float32)
    assert (other != rs).any()  # the rows tell the two apart
