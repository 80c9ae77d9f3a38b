"""The experts in bf16 and int8 on the GPU against 64-bit implementations
(expert_oracle.py): products and their gradients over ragged groups, the
activation and its gradient, int8 rows."""
import math

import pytest
import torch

import combine_count_amd as epdc
import expert_oracle as O

pytestmark = pytest.mark.gpu

KIND = {torch.bfloat16: epdc.EPDC_BF16, torch.float32: epdc.EPDC_FP32}
BF16, FP32 = torch.bfloat16, torch.float32
NAN = math.nan


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def guarded(shape, dtype, fill, value=None):
    """A tensor in the middle of a larger one that holds `fill` on both sides (the sides stay 16-byte aligned)."""
    n = math.prod(shape)
    pad = 64
    buf = torch.empty(n + 2 * pad, device="cuda", dtype=dtype)
    if dtype == torch.int8:
        buf.fill_(int(fill) if fill == fill else 99)
    else:
        buf.fill_(fill)
    t = buf[pad:pad + n].view(*shape)
    if value is not None:
        t.copy_(value)
    return t


def whole(t):
    """What lies around a guarded tensor."""
    n = t.numel()
    return torch.as_strided(t, (64,), (1,), t.storage_offset() - 64), torch.as_strided(t, (64,), (1,), t.storage_offset() + n)


def guards_hold(t, fill):
    for side in whole(t):
        assert (torch.isnan(side).all() if fill != fill else (side == fill).all())


def offsets_of(sizes, first=0):
    o = [first]
    for s in sizes:
        o.append(o[-1] + s)
    return o


def check(got, ref, bound, what):
    got = got.double()
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    bad = ~same & ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), [(i, got[tuple(i)].item(), ref[tuple(i)].item(), bound[tuple(i)].item())
                                                 for i in bad.nonzero()[:3].tolist()])


# name: (group sizes, first offset, entries behind the last group)
GROUPS = {
    "one entry": ([1], 0, 0),
    "no entry": ([0, 0], 0, 3),
    "empty groups": ([0, 5, 0, 0, 70, 0], 0, 2),
    "ragged": ([3, 129, 1, 64, 40], 2, 5),
    "many experts": ([1, 0, 2] * 30, 1, 1),
    "a long group": ([300, 17], 0, 1),
}


class Case:
    """rows, weights and lists of one product, what no call may read or write filled with NaN."""

    def __init__(self, groups, N, H, gather, weighted, seed, transposed=False, codes=False):
        sizes, first, behind = GROUPS[groups]
        g = _gen(seed)
        self.E, self.N, self.H = len(sizes), N, H
        self.offsets = offsets_of(sizes, first)
        self.n = self.offsets[-1] + behind
        self.off = torch.tensor(self.offsets, dtype=torch.int32, device="cuda")
        self.R = max(1, self.n // 2) if gather else self.n
        inner = N if transposed else H
        self.row = None
        if gather:
            self.row = torch.randint(self.R, (self.n,), device="cuda", generator=g, dtype=torch.int32)
            self.row[::7] = -1
            self.row[3::11] = self.R
        if codes:
            self.x = guarded((self.R, inner), torch.int8, 99,
                             torch.randint(-127, 128, (self.R, inner), device="cuda", generator=g, dtype=torch.int8))
            self.b = guarded((self.E, N, H), torch.int8, 99,
                             torch.randint(-128, 128, (self.E, N, H), device="cuda", generator=g, dtype=torch.int16).to(torch.int8))
            self.sx = guarded((self.R,), FP32, NAN, torch.rand(self.R, device="cuda", generator=g))
            self.sb = guarded((self.E, N), FP32, NAN, torch.rand(self.E, N, device="cuda", generator=g))
        else:
            self.x = guarded((self.R, inner), BF16, NAN, torch.randn(self.R, inner, device="cuda", generator=g))
            self.b = guarded((self.E, N, H), BF16, NAN, torch.randn(self.E, N, H, device="cuda", generator=g))
        self.w = None
        if weighted:
            self.w = torch.randn(self.n, device="cuda", generator=g)
            if self.n > 7:
                self.w[7] = math.inf if gather and self.row[7] < 0 else 2.0  # of a row that is not there


SHAPES = [(8, 8), (24, 40), (136, 72), (200, 264), (264, 1000), (512, 64), (72, 520)]


@pytest.mark.parametrize("out_dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,H", SHAPES)
@pytest.mark.parametrize("groups", list(GROUPS))
def test_product_bf16(groups, N, H, out_dtype):
    for gather, weighted in ((False, False), (True, True)):
        c = Case(groups, N, H, gather, weighted, seed=N * 7 + H)
        out = guarded((c.n, N), out_dtype, 5.0)
        out.fill_(5.0)
        ref, size = O.product(c.x, c.offsets, c.row, c.w, c.b, c.n, out)
        epdc.epdc_expert_linear(c.E, N, H, c.n, c.R, c.x, c.off, c.row, c.w, c.b, out, KIND[out_dtype])
        torch.cuda.synchronize()
        check(out, ref, O.product_bound(ref, size, H, out_dtype), (groups, gather))
        guards_hold(out, 5.0)


@pytest.mark.parametrize("N", [4, 12, 100])
def test_product_fp32_columns_by_four(N):
    c = Case("ragged", N, 48, True, True, seed=N)
    out = guarded((c.n, N), FP32, 5.0)
    out.fill_(5.0)
    ref, size = O.product(c.x, c.offsets, c.row, c.w, c.b, c.n, out)
    epdc.epdc_expert_linear(c.E, N, 48, c.n, c.R, c.x, c.off, c.row, c.w, c.b, out, epdc.EPDC_FP32)
    check(out, ref, O.product_bound(ref, size, 48, FP32), N)
    c = Case("ragged", N, 48, True, True, seed=N, codes=True)
    out.fill_(5.0)
    ref, _ = O.product(c.x, c.offsets, c.row, c.w, c.b, c.n, out, c.sx, c.sb)
    epdc.epdc_expert_linear_int(c.E, N, 48, c.n, c.R, c.x, c.sx, c.off, c.row, c.w, c.b, c.sb, out, epdc.EPDC_FP32)
    check(out, ref, O.int8_bound(ref, FP32), N)
    guards_hold(out, 5.0)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,H", SHAPES)
@pytest.mark.parametrize("groups", list(GROUPS))
def test_rows_grad(groups, N, H, dtype):
    for gather, weighted in ((False, False), (True, True)):
        c = Case(groups, N, H, gather, weighted, seed=N + 5 * H, transposed=True)
        out = guarded((c.n, H), dtype, 5.0)
        out.fill_(5.0)
        ref, size = O.product(c.x, c.offsets, c.row, c.w, c.b, c.n, out, transposed=True)
        epdc.epdc_expert_rows_grad(c.E, N, H, c.n, c.R, c.x, c.off, c.row, c.w, c.b, out, KIND[dtype])
        torch.cuda.synchronize()
        check(out, ref, O.product_bound(ref, size, N, dtype), (groups, gather))
        guards_hold(out, 5.0)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,H", SHAPES)
@pytest.mark.parametrize("groups", list(GROUPS))
def test_weights_grad(groups, N, H, dtype):
    for gather, base in ((False, None), (True, "apart"), (True, "same")):
        c = Case(groups, N, H, gather, False, seed=3 * N + H)
        g = _gen(N + H)
        D = c.n + 3 if gather else c.n
        d = guarded((D, N), BF16, NAN, torch.randn(D, N, device="cuda", generator=g))
        out_row = None
        if gather:
            out_row = torch.randperm(D, device="cuda", generator=g)[:c.n].to(torch.int32)
            out_row[5::13] = -2
            out_row[6::17] = D
        out = guarded((c.E, N, H), dtype, 5.0)
        out.fill_(5.0)
        b = None
        if base:
            b = torch.randn(c.E, N, H, device="cuda", generator=g).to(dtype)
            if base == "same":
                out.copy_(b)
        ref, size = O.weights_grad(d, out_row, c.x, c.row, c.offsets, c.n, c.E, b)
        epdc.epdc_expert_weights_grad(c.E, N, H, c.n, D, d, out_row, c.R, c.x, c.row, c.off, out if base == "same" else b, out,
                                      KIND[dtype])
        torch.cuda.synchronize()
        terms = max(hi - lo for lo, hi in O.groups_of(c.offsets, c.n))
        check(out, ref, O.product_bound(ref, size, terms, dtype), (groups, gather, base))
        guards_hold(out, 5.0)


@pytest.mark.parametrize("out_dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,H", [(8, 16), (24, 48), (136, 80), (200, 272), (264, 1008), (512, 64), (72, 528)])
@pytest.mark.parametrize("groups", list(GROUPS))
def test_product_int8(groups, N, H, out_dtype):
    for gather, weighted in ((False, False), (True, True)):
        c = Case(groups, N, H, gather, weighted, seed=N * 3 + H, codes=True)
        out = guarded((c.n, N), out_dtype, 5.0)
        out.fill_(5.0)
        ref, _ = O.product(c.x, c.offsets, c.row, c.w, c.b, c.n, out, c.sx, c.sb)
        epdc.epdc_expert_linear_int(c.E, N, H, c.n, c.R, c.x, c.sx, c.off, c.row, c.w, c.b, c.sb, out, KIND[out_dtype])
        torch.cuda.synchronize()
        check(out, ref, O.int8_bound(ref, out_dtype), (groups, gather))
        guards_hold(out, 5.0)


def test_int8_sums_are_exact_at_the_largest_row():
    """All codes -128: the sum of a row of EPDC_MAX_EXPERT_DIM comes within 2^18 of 2^31."""
    H = epdc.EPDC_MAX_EXPERT_DIM
    x = torch.full((5, H), -128, dtype=torch.int8, device="cuda")
    b = torch.full((1, 8, H), -128, dtype=torch.int8, device="cuda")
    b[0, 1] = 127
    one = torch.ones(8, device="cuda")
    out = torch.zeros(5, 8, device="cuda")
    off = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    epdc.epdc_expert_linear_int(1, 8, H, 5, 5, x, one, off, None, None, b, one, out, epdc.EPDC_FP32)
    ref = torch.full((5, 8), 16384.0 * H, dtype=torch.float64, device="cuda")
    ref[:, 1] = -128.0 * 127.0 * H
    assert torch.equal(out, ref.float())


def test_offsets_that_do_not_ascend():
    """A group ends at the smallest offset behind its start's: no entry is in two groups, nothing past the array."""
    N, H, n = 40, 72, 90
    g = _gen(4)
    offsets = [0, 30, 20, 200, 60, 85]
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x = torch.randn(n, H, device="cuda", generator=g).to(BF16)
    b = torch.randn(5, N, H, device="cuda", generator=g).to(BF16)
    out = torch.full((n, N), 5.0, device="cuda")
    ref, size = O.product(x, offsets, None, None, b, n, out)
    epdc.epdc_expert_linear(5, N, H, n, n, x, off, None, None, b, out, epdc.EPDC_FP32)
    check(out, ref, O.product_bound(ref, size, H, FP32), "product")
    d = torch.randn(n, N, device="cuda", generator=g).to(BF16)
    dx = torch.full((n, H), 5.0, device="cuda")
    ref, size = O.product(d, offsets, None, None, b, n, dx, transposed=True)
    epdc.epdc_expert_rows_grad(5, N, H, n, n, d, off, None, None, b, dx, epdc.EPDC_FP32)
    check(dx, ref, O.product_bound(ref, size, N, FP32), "rows")
    dw = torch.full((5, N, H), 5.0, device="cuda")
    ref, size = O.weights_grad(d, None, x, None, offsets, n, 5, None)
    epdc.epdc_expert_weights_grad(5, N, H, n, n, d, None, n, x, None, off, None, dw, epdc.EPDC_FP32)
    check(dw, ref, O.product_bound(ref, size, n, FP32), "weights")


def test_a_rows_nan_stays_in_its_row():
    """NaN and infinities in a row, in a weight's row and in rows that nobody takes reach no other output."""
    N, H = 72, 104
    c = Case("ragged", N, H, True, False, seed=8)
    used = [r for lo, hi in O.groups_of(c.offsets, c.n) for r in c.row[lo:hi].tolist() if 0 <= r < c.R]
    c.x[used[0]] = NAN
    c.x[used[1], 5] = math.inf
    c.b[1, 3] = NAN
    out = torch.full((c.n, N), 5.0, device="cuda")
    ref, size = O.product(c.x, c.offsets, c.row, None, c.b, c.n, out)
    epdc.epdc_expert_linear(c.E, N, H, c.n, c.R, c.x, c.off, c.row, None, c.b, out, epdc.EPDC_FP32)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(out), fine) and fine.any() and not fine.all()
    check(out[fine], ref[fine], O.product_bound(ref, size, H, FP32)[fine], "product")
    # the weights' gradient: a NaN in an entry's row reaches that expert's column only
    x = torch.randn(c.R, H, device="cuda", generator=_gen(1)).to(BF16)
    d = torch.randn(c.n, N, device="cuda", generator=_gen(2)).to(BF16)
    lo, hi = O.groups_of(c.offsets, c.n)[1]
    at = next(i for i in range(lo, hi) if 0 <= int(c.row[i]) < c.R)
    d[at, 9] = NAN
    dw = torch.full((c.E, N, H), 5.0, device="cuda")
    ref, size = O.weights_grad(d, None, x, c.row, c.offsets, c.n, c.E, None)
    epdc.epdc_expert_weights_grad(c.E, N, H, c.n, c.n, d, None, c.R, x, c.row, c.off, None, dw, epdc.EPDC_FP32)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(dw), fine) and int((~fine).sum()) == H
    check(dw[fine], ref[fine], O.product_bound(ref, size, c.n, FP32)[fine], "weights")


def test_gradients_are_the_products_adjoints():
    """<out(x + d) - out(x), g> = <d, rows' gradient> and the same for the weights: the product is linear, so the
    difference is the derivative at any step; what is left is the fp32 sums' rounding."""
    N, H = 136, 264
    c = Case("a long group", N, H, False, True, seed=21)
    lo, hi = c.offsets[0], c.offsets[-1]
    gen = _gen(22)
    g = torch.randn(c.n, N, device="cuda", generator=gen).to(BF16)
    g[hi:] = 0
    d = torch.randn(c.n, H, device="cuda", generator=gen).to(BF16)
    x2 = (c.x.float() + d.float()).to(BF16)  # x2 - x is the step, whatever the rounding
    step = x2.double() - c.x.double()
    outs = []
    for x in (c.x, x2):
        o = torch.zeros(c.n, N, device="cuda")
        epdc.epdc_expert_linear(c.E, N, H, c.n, c.R, x, c.off, None, c.w, c.b, o, epdc.EPDC_FP32)
        outs.append(o.double())
    dx = torch.zeros(c.n, H, device="cuda")
    epdc.epdc_expert_rows_grad(c.E, N, H, c.n, c.n, g, c.off, None, c.w, c.b, dx, epdc.EPDC_FP32)
    left, right = ((outs[1] - outs[0]) * g.double()).sum(1)[lo:hi], (step * dx.double()).sum(1)[lo:hi]  # of an entry
    _, s0 = O.product(c.x, c.offsets, None, c.w, c.b, c.n, outs[0])
    _, s1 = O.product(x2, c.offsets, None, c.w, c.b, c.n, outs[0])
    _, s2 = O.product(g, c.offsets, None, c.w, c.b, c.n, dx, transposed=True)
    room = (H + 4) * 2.0 ** -23 * ((s0 + s1) * g.double().abs()).sum(1) + (N + 4) * 2.0 ** -23 * (s2 * step.abs()).sum(1)
    assert ((left - right).abs() <= room[lo:hi]).all() and right.abs().median() > 4 * room.median()
    # the weights: out with w = 1 is linear in them too
    b2 = (c.b.float() + torch.randn(c.b.shape, device="cuda", generator=gen)).to(BF16)
    outs, sizes = [], []
    for b in (c.b, b2):
        o = torch.zeros(c.n, N, device="cuda")
        epdc.epdc_expert_linear(c.E, N, H, c.n, c.R, c.x, c.off, None, None, b, o, epdc.EPDC_FP32)
        outs.append(o.double())
        sizes.append(O.product(c.x, c.offsets, None, None, b, c.n, o)[1])
    dw = torch.zeros(c.E, N, H, device="cuda")
    epdc.epdc_expert_weights_grad(c.E, N, H, c.n, c.n, g, None, c.R, c.x, None, c.off, None, dw, epdc.EPDC_FP32)
    step = b2.double() - c.b.double()
    _, s2 = O.weights_grad(g, None, c.x, None, c.offsets, c.n, c.E, None)
    for e, (lo, hi) in enumerate(O.groups_of(c.offsets, c.n)):  # of an expert's column
        left, right = ((outs[1] - outs[0]) * g.double())[lo:hi].sum(0), (step[e] * dw[e].double()).sum(1)
        room = (H + 4) * 2.0 ** -23 * ((sizes[0] + sizes[1]) * g.double().abs())[lo:hi].sum(0)
        room += (hi - lo + 4) * 2.0 ** -23 * (s2[e] * step[e].abs()).sum(1)
        assert ((left - right).abs() <= room).all() and right.abs().median() > 4 * room.median()


# ---- the activation ------------------------------------------------------------------------------------------------


def _values(n, cols, g):
    h = 2.0 * torch.randn(n, 2 * cols, device="cuda", generator=g)
    h.view(-1)[::5] *= 20.0
    h.view(-1)[7::31] = 0.0
    return h


GATE_SHAPES = [(1, 8), (3, 40), (70, 256), (33, 520), (5, 2048), (2, 9000)]


@pytest.mark.parametrize("out_dtype", [BF16, FP32], ids=["to_bf16", "to_fp32"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,cols", GATE_SHAPES)
def test_gate_and_its_gradient(n, cols, dtype, out_dtype):
    g = _gen(n + cols)
    total = n + 5
    h = guarded((total, 2 * cols), dtype, NAN, _values(total, cols, g))
    d = guarded((total, cols), out_dtype, NAN, torch.randn(total, cols, device="cuda", generator=g))
    for weighted in (False, True):
        w = torch.randn(total, device="cuda", generator=g) if weighted else None
        for offsets in (None, [2, 2, 2 + n]):
            lo, hi = (0, total) if offsets is None else (offsets[0], offsets[-1])
            E = 1 if offsets is None else 2
            off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
            out = guarded((total, cols), out_dtype, 5.0)
            out.fill_(5.0)
            epdc.epdc_expert_gate(E, cols, total, KIND[dtype], h, off, w, out, KIND[out_dtype])
            ref = O.gate(h, w)
            check(out[lo:hi], ref[lo:hi], O.gate_bound(h, w, ref, out_dtype)[lo:hi], ("gate", weighted, offsets))
            assert (out[:lo] == 5).all() and (out[hi:] == 5).all()
            guards_hold(out, 5.0)
            dh = guarded((total, 2 * cols), dtype, 5.0)
            dh.fill_(5.0)
            dw = guarded((total,), FP32, 5.0)
            dw.fill_(5.0)
            epdc.epdc_expert_gate_grad(E, cols, total, KIND[dtype], h, off, w, d, KIND[out_dtype], dh, dw)
            rh, rw, size, size_w = O.gate_grad(h, w, d)
            bh, bw = O.gate_grad_bounds(h, rh, rw, size, size_w, dtype)
            check(dh[lo:hi], rh[lo:hi], bh[lo:hi], ("dH", weighted, offsets))
            check(dw[lo:hi], rw[lo:hi], bw[lo:hi], ("dw", weighted, offsets))
            for t in (dh, dw):
                assert (t[:lo] == 5).all() and (t[hi:] == 5).all()
                guards_hold(t, 5.0)
            again = torch.full_like(dh, 5.0)
            epdc.epdc_expert_gate_grad(E, cols, total, KIND[dtype], h, off, w, d, KIND[out_dtype], again, None)
            assert torch.equal(again, dh)


def test_gate_gradient_against_differences():
    """Central differences of the fp32 activation: step 2^-7, error step^2 / 6 times the third derivative (below
    1 for a gate in [-4, 4], times |u w|), and the two values' rounding over the step."""
    n, cols, step = 6, 64, 2.0 ** -7
    g = _gen(3)
    h = (torch.rand(n, 2 * cols, device="cuda", generator=g) * 8 - 4)
    h = torch.round(h * 1024) / 1024  # so that the steps are exact
    w = torch.rand(n, device="cuda", generator=g) + 0.5
    d = torch.ones(n, cols, device="cuda")
    dh, dw = torch.zeros_like(h), torch.zeros(n, device="cuda")
    epdc.epdc_expert_gate_grad(1, cols, n, epdc.EPDC_FP32, h, None, w, d, epdc.EPDC_FP32, dh, dw)

    def value(x, weights=w):
        out = torch.zeros(n, cols, device="cuda")
        epdc.epdc_expert_gate(1, cols, n, epdc.EPDC_FP32, x, None, weights, out, epdc.EPDC_FP32)
        return out.double()

    big = (h[:, cols:].abs().clamp_min(1) * w[:, None]).double()
    room = big * (step * step / 6 + 4 * 10 * 2.0 ** -24 / step)
    for part in (0, 1):
        up, down = h.clone(), h.clone()
        up[:, part * cols:(part + 1) * cols] += step
        down[:, part * cols:(part + 1) * cols] -= step
        slope = (value(up) - value(down)) / (2 * step)
        assert ((slope - dh[:, part * cols:(part + 1) * cols].double()).abs() <= room).all(), part
    slope = ((value(h, w + 0.5) - value(h, w - 0.5))).sum(1)  # linear in w
    assert ((slope - dw.double()).abs() <= 40 * 2.0 ** -24 * 4 * 4 * 2 * cols).all()


def test_gate_of_special_values():
    """Extreme gates: no overflow of the exponential reaches the result; NaN and -inf as the formula gives them."""
    vals = [0.0, -0.0, 88.0, -88.0, 100.0, -100.0, 1e30, -1e30, math.inf, -math.inf, NAN, 2.0 ** -140, -2.0 ** -140, 1.0, -1.0, 17.0]
    h = torch.zeros(1, 32, device="cuda")
    h[0, :16] = torch.tensor(vals)
    h[0, 16:] = 1.0
    out = torch.zeros(1, 16, device="cuda")
    epdc.epdc_expert_gate(1, 16, 1, epdc.EPDC_FP32, h, None, None, out, epdc.EPDC_FP32)
    g = h[:, :16].double()
    ref = g * torch.sigmoid(g)
    same = torch.isnan(ref) == torch.isnan(out)
    assert same.all() and torch.isnan(out[0, 9]) and torch.isnan(out[0, 10]) and out[0, 8] == math.inf
    fine = torch.isfinite(ref)
    assert ((out.double() - ref).abs()[fine] <= 9 * 2.0 ** -24 * ref.abs()[fine] + 2.0 ** -148 * g.abs()[fine] + 2.0 ** -149).all()


# ---- int8 rows -----------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,cols", [(1, 16), (7, 48), (70, 256), (9, 1024), (9, 1040), (5, 7168), (3, 20000)])
def test_int_quantize(n, cols, dtype):
    g = _gen(n * cols)
    W, M = 2, n + 2
    x = torch.randn(W * M, cols, device="cuda", generator=g) * torch.exp(3 * torch.randn(W * M, 1, device="cuda", generator=g))
    x = guarded((W, M, cols), dtype, NAN, x.view(W, M, cols))
    x[0, 0] = 0.0
    # halves of the maximum are exactly between two codes
    x[1, 0, :8] = torch.tensor([8.0, 4.0, -4.0, 2.0, -8.0, 1.0, 0.5, -0.25], device="cuda")
    x[1, 0, 8:] = x[1, 0, 8:].clamp(-6, 6)
    if n > 2:
        x[0, 1, 3], x[0, 2, cols - 1], x[1, 1, 0] = NAN, math.inf, -math.inf
    if dtype == FP32 and n > 4:
        x[1, 2] *= 2.0 ** -140  # subnormal, the scale a few steps of 2^-149
        x[1, 3] *= 2.0 ** -160
    for count in (None, [n, 1]):
        q = guarded((W, M, cols), torch.int8, 77)
        q.fill_(77)
        s = guarded((W, M), FP32, 5.0)
        s.fill_(5.0)
        cnt = None if count is None else torch.tensor(count, dtype=torch.int32, device="cuda")
        epdc.epdc_int_quantize(W, M, cols, KIND[dtype], x, cnt, q, s)
        for wi in range(W):
            live = M if count is None else count[wi]
            rq, rs = O.int8_rows(x[wi, :live])
            assert torch.equal(q[wi, :live].cpu(), rq), (wi, live)
            assert torch.equal(torch.nan_to_num(s[wi, :live].cpu(), nan=-1.0), torch.nan_to_num(rs, nan=-1.0))
            assert (q[wi, live:] == 77).all() and (s[wi, live:] == 5).all()
        guards_hold(q, 77)
        guards_hold(s, 5.0)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,cols", [(1, 16), (70, 256), (9, 512), (9, 528), (40, 2048), (3, 9008)])
def test_gate_int8(n, cols, dtype):
    g = _gen(n * cols + 1)
    total = n + 3
    h = guarded((total, 2 * cols), dtype, NAN, _values(total, cols, g))
    if n > 4:
        h[3] = 0.0
        h[4, 2] = NAN
        h[5, cols + 3] = math.inf
    if dtype == FP32 and n > 8:
        h[6] *= 1e25   # products beyond fp32: infinite
        h[7, :cols] *= 1e-25  # small values of large and small factors
        h[7, cols:] *= 1e20
        h[8] *= 1e-30  # below fp32's least
    for weighted in (False, True):
        w = torch.rand(total, device="cuda", generator=g) if weighted else None
        for offsets in (None, [1, 1 + n]):
            lo, hi = (0, total) if offsets is None else (offsets[0], offsets[-1])
            off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
            q = guarded((total, cols), torch.int8, 77)
            q.fill_(77)
            s = guarded((total,), FP32, 5.0)
            s.fill_(5.0)
            epdc.epdc_expert_gate_int(1, cols, total, KIND[dtype], h, off, w, q, s)
            rq, rs = O.int8_rows(O.gate(h, w).float())
            assert torch.equal(torch.nan_to_num(s[lo:hi].cpu(), nan=-1.0), torch.nan_to_num(rs[lo:hi], nan=-1.0))
            assert torch.equal(q[lo:hi].cpu(), rq[lo:hi])
            assert (q[:lo] == 77).all() and (q[hi:] == 77).all() and (s[:lo] == 5).all() and (s[hi:] == 5).all()
            guards_hold(q, 77)
            guards_hold(s, 5.0)
