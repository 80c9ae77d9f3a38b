"""Groups of more than 2^28 entries: the weights' gradient goes over them to
the end, and not past it (whole numbers, whose sums fp32 holds exactly).  And
the activation in codes of more rows than a grid has blocks for."""
import pytest
import torch

import combine_count_amd as epdc

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
N = H = 8
LONG = 2 ** 28 + 9 * 64 + 17  # entries of the long group: whole steps of 64 and a part of one
BEHIND = 40                   # entries that belong to no group
EDGE = 700                    # rows that count, at either end


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def _small(g, *shape):
    return torch.randint(-3, 4, shape, device="cuda", generator=g).to(BF16)


def _product(d, x):
    return d.double().t().contiguous() @ x.double()


def test_weights_grad_of_a_group_beyond_2_28_entries():
    """Entries in order: a short group, the long one, entries behind it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    first, n = 5, 5 + LONG
    d, x = (torch.zeros(n + BEHIND, 8, device="cuda", dtype=BF16) for _ in range(2))
    for t in (d, x):
        t[:first + EDGE], t[n - EDGE:] = _small(g, first + EDGE, 8), _small(g, EDGE + BEHIND, 8)
    out = torch.full((2, N, H), 5.0, device="cuda")
    off = torch.tensor([0, first, n], dtype=torch.int32, device="cuda")
    epdc.epdc_expert_weights_grad(2, N, H, n + BEHIND, n + BEHIND, d, None, n + BEHIND, x, None, off, None, out, epdc.EPDC_FP32)
    torch.cuda.synchronize()
    assert torch.equal(out[0].double(), _product(d[:first], x[:first]))
    ref = _product(d[first:first + EDGE], x[first:first + EDGE]) + _product(d[n - EDGE:n], x[n - EDGE:n])
    assert torch.equal(out[1].double(), ref)


def test_weights_grad_of_gathered_entries_beyond_2_28():
    """Both lists given: the last step's places behind the group's end are no entries."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    rows = 33
    d, x = _small(g, rows, N), _small(g, rows, H)
    d[0] = 0  # what all entries but those at the ends take
    lists = []
    for _ in range(2):
        t = torch.zeros(LONG + BEHIND, dtype=torch.int32, device="cuda")
        for part in (t[:EDGE], t[LONG - EDGE:]):
            part.copy_(torch.randint(1, rows, (part.numel(),), device="cuda", generator=g))
        lists.append(t)
    out_row, row = lists
    row[3], row[LONG - 2], out_row[LONG - 5] = -1, rows, rows + 7  # entries that add nothing
    out = torch.full((1, N, H), 5.0, device="cuda")
    off = torch.tensor([0, LONG], dtype=torch.int32, device="cuda")
    epdc.epdc_expert_weights_grad(1, N, H, LONG + BEHIND, rows, d, out_row, rows, x, row, off, None, out, epdc.EPDC_FP32)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(EDGE, device="cuda"), torch.arange(LONG - EDGE, LONG, device="cuda")])
    o, r = out_row[at].long(), row[at].long()
    there = (o < rows) & (r >= 0) & (r < rows)
    assert torch.equal(out[0].double(), _product(d[o[there]], x[r[there]]))


def test_gate_int_of_more_rows_than_a_grid_has_blocks():
    """Rows beyond 2^23 blocks of four: the blocks go on to them."""
    import expert_oracle as O
    n, last, cols = 34_000_001, 50, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    h = torch.zeros(n, 2 * cols, device="cuda", dtype=BF16)
    for part in (slice(0, last), slice(n - last, n)):
        h[part] = 2 * torch.randn(last, 2 * cols, device="cuda", generator=g)
    q, s = torch.full((n, cols), 7, device="cuda", dtype=torch.int8), torch.full((n,), 5.0, device="cuda")
    epdc.epdc_expert_gate_int(1, cols, n, epdc.EPDC_BF16, h, None, None, q, s)
    for part in (slice(0, last), slice(n - last, n)):
        rq, rs = O.int8_rows(O.gate(h[part], None).float())
        assert torch.equal(q[part].cpu(), rq) and torch.equal(s[part].cpu(), rs)
    assert (q[last:-last] == 0).all() and (s[last:-last] == 0).all()
