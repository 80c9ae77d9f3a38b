"""The activation of more elements than a grid has blocks for (2^23 blocks of
4096): the blocks go on to those behind.  200 GB of rows of which the last few are
in the groups, the only ones that are read and written."""
import pytest
import torch

import combine_count_amd as epdc
import expert_oracle as O

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_gate_beyond_a_grids_blocks():
    cols, live = 8192, 30
    n = 2 ** 23 * 4096 // cols + 100  # rows; those behind the first grid are 100
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 6 * n * cols + 2 ** 30:
        pytest.skip("needs 207 GB of free memory")
    h, out = torch.empty(n, 2 * cols, device="cuda", dtype=BF16), torch.empty(n, cols, device="cuda", dtype=BF16)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    h[-live:] = torch.randn(live, 2 * cols, device="cuda", generator=g)
    out[-live - 5:] = 5.0
    off = torch.tensor([n - live, n - 2], dtype=torch.int32, device="cuda")
    epdc.epdc_expert_gate(1, cols, n, epdc.EPDC_BF16, h, off, None, out, epdc.EPDC_BF16)
    part = h[-live:-2]
    ref = O.gate(part, None)
    assert ((out[-live:-2].double() - ref).abs() <= O.gate_bound(part, None, ref, BF16)).all()
    assert (out[-live - 5:-live] == 5).all() and (out[-2:] == 5).all()
    del h, out, part
    torch.cuda.empty_cache()
