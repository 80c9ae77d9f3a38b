"""The experts in bf16 and int8 where offsets pass 32 bits: rows, weights,
gradients and activations beyond 4 GB, of which the ends are used."""
import pytest
import torch

import combine_count_amd as epdc
import expert_oracle as O

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
H, N = 7168, 512


def _near(got, ref, bound):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def _lists(rows, n, g):
    """Entries at both ends of the rows, of the first, a middle and the last expert."""
    row = torch.cat([torch.arange(n // 2, device="cuda"), rows - 1 - torch.arange(n - n // 2, device="cuda")])
    return row[torch.randperm(n, device="cuda", generator=g)].to(torch.int32)


@pytest.mark.parametrize("rows_grad", [False, True], ids=["product", "rows_grad"])
def test_rows_and_weights_beyond_4_gb(rows_grad):
    g = _gen(1)
    R, n, E = 300001, 90, 700  # rows 4.3 GB, weights 5.1 GB
    cols = H if rows_grad else N  # the product's columns; the other is its row length
    inner = N if rows_grad else H
    x = torch.zeros(R, H, device="cuda", dtype=BF16)
    x = x.view(-1)[:R * H].view(R, H)
    x[:n], x[-n:] = torch.randn(n, H, device="cuda", generator=g), torch.randn(n, H, device="cuda", generator=g)
    b = torch.zeros(E, N * H, device="cuda", dtype=BF16)
    used = [0, 333, E - 1]
    for e in used:
        b[e] = torch.randn(N * H, device="cuda", generator=g)
    sizes = torch.zeros(E, dtype=torch.int64)
    sizes[used] = 30
    off = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)])
    row = _lists(R, n, g)
    out = torch.zeros(n, N, device="cuda")
    # rows of H summed over H: the product takes [E][N][H], the rows' gradient [E][H (its columns)][N (its row length)]
    d = off.to(torch.int32).cuda()
    if rows_grad:
        b = b.view(E, H, N)
        epdc.epdc_expert_rows_grad(E, cols, inner, n, R, x, d, row, None, b, out, epdc.EPDC_FP32)
    else:
        b = b.view(E, N, H)
        epdc.epdc_expert_linear(E, cols, inner, n, R, x, d, row, None, b, out, epdc.EPDC_FP32)
    ref, size = O.product(x, off.tolist(), row, None, b, n, out, transposed=rows_grad)
    _near(out, ref, O.product_bound(ref, size, H, torch.float32))


def test_weights_grad_beyond_4_gb():
    g = _gen(2)
    R, n, E = 300001, 90, 700  # rows 4.3 GB, gradients 5.1 GB
    x = torch.zeros(R, H, device="cuda", dtype=BF16)
    x[:n], x[-n:] = torch.randn(n, H, device="cuda", generator=g), torch.randn(n, H, device="cuda", generator=g)
    d = torch.randn(n, N, device="cuda", generator=g).to(BF16)
    used = [0, 333, E - 1]
    sizes = torch.zeros(E, dtype=torch.int64)
    sizes[used] = 30
    off = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)])
    row = _lists(R, n, g)
    dw = torch.full((E, N, H), 5.0, device="cuda", dtype=BF16)
    epdc.epdc_expert_weights_grad(E, N, H, n, n, d, None, R, x, row, off.to(torch.int32).cuda(), None, dw, epdc.EPDC_BF16)
    for e in range(0, E, 50):
        if e not in used:
            assert (dw[e] == 0).all()
    for i, e in enumerate(used):
        lo = 30 * i
        a, r = d[lo:lo + 30].double().t().contiguous(), x[row[lo:lo + 30].long()].double()
        ref, size = a @ r, a.abs() @ r.abs()
        _near(dw[e], ref, O.product_bound(ref, size, 30, BF16))


def test_int8_weights_beyond_4_gb():
    g = _gen(3)
    n, E, h, cols = 40, 300, 7168, 2048  # 4.4 GB
    b = torch.zeros(E, cols, h, device="cuda", dtype=torch.int8)
    for e in (0, E - 1):
        b[e] = torch.randint(-127, 128, (cols, h), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
    sb = torch.rand(E, cols, device="cuda", generator=g)
    x = torch.randint(-127, 128, (n, h), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
    sx = torch.rand(n, device="cuda", generator=g)
    off = [0] + [20] * (E - 1) + [n]
    out = torch.zeros(n, cols, device="cuda")
    epdc.epdc_expert_linear_int(E, cols, h, n, n, x, sx, torch.tensor(off, dtype=torch.int32, device="cuda"), None, None, b, sb,
                                out, epdc.EPDC_FP32)
    ref, _ = O.product(x, off, None, None, b, n, out, sx, sb)
    _near(out, ref, O.int8_bound(ref, torch.float32))


def test_gates_beyond_4_gb():
    n, F = 150001, 8192  # h 4.9 GB
    h = torch.zeros(n, 2 * F, device="cuda", dtype=BF16)
    g = _gen(4)
    last = 20
    h[-last:] = 2 * torch.randn(last, 2 * F, device="cuda", generator=g)
    off = torch.tensor([n - last, n], dtype=torch.int32, device="cuda")
    w = torch.rand(n, device="cuda", generator=g)
    out = torch.zeros(n, F, device="cuda", dtype=BF16)
    epdc.epdc_expert_gate(1, F, n, epdc.EPDC_BF16, h, off, w, out, epdc.EPDC_BF16)
    ref = O.gate(h[-last:], w[-last:])
    _near(out[-last:], ref, O.gate_bound(h[-last:], w[-last:], ref, BF16))
    assert (out[:-last:1000] == 0).all()
    q, s = torch.zeros(n, F, device="cuda", dtype=torch.int8), torch.zeros(n, device="cuda")
    epdc.epdc_expert_gate_int(1, F, n, epdc.EPDC_BF16, h, off, w, q, s)
    rq, rs = O.int8_rows(ref.float())
    assert torch.equal(q[-last:].cpu(), rq) and torch.equal(s[-last:].cpu(), rs)
    d, dh, dw = out, torch.zeros_like(h), torch.zeros(n, device="cuda")
    epdc.epdc_expert_gate_grad(1, F, n, epdc.EPDC_BF16, h, off, w, d, epdc.EPDC_BF16, dh, dw)
    rh, rw, size, size_w = O.gate_grad(h[-last:], w[-last:], d[-last:])
    bh, bw = O.gate_grad_bounds(h[-last:], rh, rw, size, size_w, BF16)
    _near(dh[-last:], rh, bh)
    _near(dw[-last:], rw, bw)
    # int8 rows of the same array
    epdc.epdc_int_quantize(1, n, 2 * F, epdc.EPDC_BF16, h, None, torch.empty(n, 2 * F, device="cuda", dtype=torch.int8), s)
    assert (s[:-last:1000] == 0).all() and (s[-last:] > 0).all()


def test_no_rows_at_all():
    """numRows 0: every entry is a row of +0, every gradient 0 or the base."""
    E, n, cols, h = 3, 50, 136, 72
    off = torch.tensor([0, 20, 20, n], dtype=torch.int32, device="cuda")
    b = torch.randn(E, cols, h, device="cuda").to(BF16)
    out = torch.full((n, cols), 5.0, device="cuda")
    epdc.epdc_expert_linear(E, cols, h, n, 0, None, off, None, None, b, out, epdc.EPDC_FP32)
    assert torch.equal(out, torch.zeros_like(out)) and not torch.signbit(out).any()
    dx = torch.full((n, h), 5.0, device="cuda")
    epdc.epdc_expert_rows_grad(E, cols, h, n, 0, None, off, None, None, b, dx, epdc.EPDC_FP32)
    assert torch.equal(dx, torch.zeros_like(dx))
    base = torch.randn(E, cols, h, device="cuda")
    d = torch.randn(n, cols, device="cuda").to(BF16)
    for bs, want in ((None, torch.zeros_like(base)), (base, base)):
        dw = torch.full((E, cols, h), 5.0, device="cuda")
        epdc.epdc_expert_weights_grad(E, cols, h, n, n, d, None, 0, None, None, off, bs, dw, epdc.EPDC_FP32)
        assert torch.equal(dw, want)
    one = torch.ones(E * cols, device="cuda")
    q = torch.ones(E, cols, 80, device="cuda", dtype=torch.int8)
    out = torch.full((n, cols), 5.0, device="cuda")
    epdc.epdc_expert_linear_int(E, cols, 80, n, 0, None, None, off, None, None, q, one, out, epdc.EPDC_FP32)
    assert torch.equal(out, torch.zeros_like(out))
    # and no entries
    dw = torch.full((E, cols, h), 5.0, device="cuda")
    epdc.epdc_expert_weights_grad(E, cols, h, 0, n, d, None, n, torch.randn(n, h, device="cuda").to(BF16), None, off, None, dw,
                                  epdc.EPDC_FP32)
    assert torch.equal(dw, torch.zeros_like(dw))


def test_more_rows_than_a_grid_has_blocks():
    """Rows beyond 2^23 blocks of four: the blocks go on to them."""
    n, last, cols = 34_000_001, 50, 16
    g = _gen(6)
    x = torch.zeros(n, cols, device="cuda", dtype=BF16)
    x[-last:] = torch.randn(last, cols, device="cuda", generator=g)
    x[:last] = torch.randn(last, cols, device="cuda", generator=g)
    q, s = torch.full((n, cols), 7, device="cuda", dtype=torch.int8), torch.full((n,), 5.0, device="cuda")
    epdc.epdc_int_quantize(1, n, cols, epdc.EPDC_BF16, x, None, q, s)
    for part in (slice(0, last), slice(n - last, n)):
        rq, rs = O.int8_rows(x[part])
        assert torch.equal(q[part].cpu(), rq) and torch.equal(s[part].cpu(), rs)
    assert (q[last:-last] == 0).all() and (s[last:-last] == 0).all()
    # the same array as rows of two halves of eight
    d, dh, dw = torch.ones(n, 8, device="cuda", dtype=BF16), torch.full_like(x, 5.0), torch.full((n,), 5.0, device="cuda")
    epdc.epdc_expert_gate_grad(1, 8, n, epdc.EPDC_BF16, x, None, None, d, epdc.EPDC_BF16, dh, dw)
    for part in (slice(0, last), slice(n - last, n)):
        rh, rw, size, size_w = O.gate_grad(x[part], None, d[part])
        bh, bw = O.gate_grad_bounds(x[part], rh, rw, size, size_w, BF16)
        _near(dh[part], rh, bh)
        _near(dw[part], rw, bw)
    assert (dh[last:-last] == 0).all() and (dw[last:-last] == 0).all()
