"""A sparse layer's training step and its int8 forward pass through the
library's calls: route, dispatch, group, product, activation with the routing
weight, product, combine, and back through all of them; each call against the
64-bit formula on the inputs that it was given, the whole against automatic
differentiation in 64 bits.  Eager, captured and replayed, on two streams."""
import pytest
import torch

import combine_count_amd as epdc
import expert_oracle as O

pytestmark = pytest.mark.gpu

BF16, FP32 = epdc.EPDC_BF16, epdc.EPDC_FP32
T, W, EPR, K, H, F = 70, 4, 3, 3, 136, 72
E, M = W * EPR, T
DEV = "cuda"


def _bf(*shape, g, scale=1.0):
    return (scale * torch.randn(*shape, device=DEV, generator=g)).bfloat16()


class Layer:
    """Buffers and calls of one step, in order."""

    def __init__(self, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.cfg = epdc.EpCfg(W, H, M, EPR, K, BF16, 1, 0)
        self.rcfg = epdc.RouteCfg(E, K, FP32, epdc.EPDC_SOFTMAX, renormalize=1)
        self.x, self.logits = _bf(T, H, g=g), torch.randn(T, E, device=DEV, generator=g)
        self.w1, self.w2 = _bf(E, 2 * F, H, g=g, scale=H ** -0.5), _bf(E, H, F, g=g, scale=F ** -0.5)
        self.dy = _bf(T, H, g=g)
        i32 = lambda *s: torch.full(s, -7, dtype=torch.int32, device=DEV)
        f32 = lambda *s: torch.full(s, -7.0, device=DEV)
        bf = lambda *s: torch.full(s, -7.0, device=DEV, dtype=torch.bfloat16)
        n = self.n = W * M * K
        self.ids, self.weights = i32(T, K), f32(T, K)
        self.buf, self.back = epdc.DispatchBuffers(self.cfg), epdc.DispatchBuffers(self.cfg)
        self.offsets, self.row, self.wgt, self.of = i32(E + 1), i32(n), f32(n), i32(W, M, K)
        self.gscratch = torch.zeros(epdc.epdc_group_scratch_bytes(self.cfg, -1) // 4 + 4, dtype=torch.int32, device=DEV)
        self.h1, self.a, self.y2 = bf(n, 2 * F), bf(n, F), bf(n, H)
        self.yrow, self.y = bf(W * M, H), bf(T, H)
        self.da, self.dh1, self.dwgt = bf(n, F), bf(n, 2 * F), f32(n)
        self.dx2, self.dxrow, self.dx = bf(n, H), bf(W * M, H), bf(T, H)
        self.dw1, self.dw2 = f32(E, 2 * F, H), f32(E, H, F)
        # rows of a window summed over its entries: entryOf is a sendMap into them
        self.sum = epdc.EpCfg(1, H, n, K, K, BF16, 0, 0)
        self.plain = epdc.EpCfg(W, H, M, EPR, K, BF16, 0, 0)
        b, k = self.buf, self.back
        self.calls = [
            epdc.prepare_route(self.rcfg, T, self.logits, None, self.ids, self.weights),
            epdc.prepare_dispatch(self.cfg, T, self.x, self.ids, self.weights, None, b.recvX, b.recvTokIdx, b.recvExpertIds,
                                  b.recvWeights, None, b.recvCount, b.sendMap, b.scratch),
            epdc.prepare_group_experts(self.cfg, -1, b.recvExpertIds, b.recvWeights, b.recvCount, self.offsets, self.row,
                                       self.wgt, self.of, self.gscratch),
            epdc.prepare_expert_linear(E, 2 * F, H, n, W * M, b.recvX, self.offsets, self.row, None, self.w1, self.h1, BF16),
            epdc.prepare_expert_gate(E, F, n, BF16, self.h1, self.offsets, self.wgt, self.a, BF16),
            epdc.prepare_expert_linear(E, H, F, n, n, self.a, self.offsets, None, None, self.w2, self.y2, BF16),
            epdc.prepare_combine(self.sum, W * M, self.y2, None, None, self.of, self.yrow),
            epdc.prepare_combine(self.plain, T, self.yrow, None, None, b.sendMap, self.y),
            # back: the tokens' gradients go the same way as the tokens, every row to its entries
            epdc.prepare_dispatch(self.cfg, T, self.dy, self.ids, self.weights, None, k.recvX, k.recvTokIdx, k.recvExpertIds,
                                  k.recvWeights, None, k.recvCount, k.sendMap, k.scratch),
            epdc.prepare_expert_weights_grad(E, H, F, n, W * M, k.recvX, self.row, n, self.a, None, self.offsets, None,
                                             self.dw2, FP32),
            epdc.prepare_expert_rows_grad(E, H, F, n, W * M, k.recvX, self.offsets, self.row, None, self.w2, self.da, BF16),
            epdc.prepare_expert_gate_grad(E, F, n, BF16, self.h1, self.offsets, self.wgt, self.da, BF16, self.dh1, self.dwgt),
            epdc.prepare_expert_weights_grad(E, 2 * F, H, n, n, self.dh1, None, W * M, b.recvX, self.row, self.offsets, None,
                                             self.dw1, FP32),
            epdc.prepare_expert_rows_grad(E, 2 * F, H, n, n, self.dh1, self.offsets, None, None, self.w1, self.dx2, BF16),
            epdc.prepare_combine(self.sum, W * M, self.dx2, None, None, self.of, self.dxrow),
            epdc.prepare_combine(self.plain, T, self.dxrow, None, None, b.sendMap, self.dx),
        ]

    def run(self):
        for call in self.calls:
            call()

    def results(self):
        n = int(self.offsets[-1])
        return {"y": self.y, "dx": self.dx, "dw1": self.dw1, "dw2": self.dw2, "dwgt": self.dwgt[:n], "h1": self.h1[:n],
                "dh1": self.dh1[:n], "ids": self.ids}


def _near(got, ref, bound):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


def _check_calls(s):
    """Every call against its formula, on the inputs that it read."""
    b, n = s.buf, s.n
    o = s.offsets.tolist()
    live = o[-1]
    assert 0 < live <= T * K
    x = b.recvX.view(W * M, H)
    ref, size = O.product(x, o, s.row, None, s.w1, n, s.h1)
    _near(s.h1[:live], ref[:live], O.product_bound(ref, size, H, torch.bfloat16)[:live])
    ref = O.gate(s.h1[:live], s.wgt[:live])
    _near(s.a[:live], ref, O.gate_bound(s.h1[:live], s.wgt[:live], ref, torch.bfloat16))
    ref, size = O.product(s.a, o, None, None, s.w2, n, s.y2)
    _near(s.y2[:live], ref[:live], O.product_bound(ref, size, F, torch.bfloat16)[:live])
    dy = s.back.recvX.view(W * M, H)
    ref, size = O.weights_grad(dy, s.row, s.a, None, o, n, E, None)
    _near(s.dw2, ref, O.product_bound(ref, size, live, torch.float32))
    ref, size = O.product(dy, o, s.row, None, s.w2, n, s.da, transposed=True)
    _near(s.da[:live], ref[:live], O.product_bound(ref, size, H, torch.bfloat16)[:live])
    dh, dw, size, size_w = O.gate_grad(s.h1[:live], s.wgt[:live], s.da[:live])
    bh, bw = O.gate_grad_bounds(s.h1[:live], dh, dw, size, size_w, torch.bfloat16)
    _near(s.dh1[:live], dh, bh)
    _near(s.dwgt[:live], dw, bw)
    ref, size = O.weights_grad(s.dh1, None, x, s.row, o, n, E, None)
    _near(s.dw1, ref, O.product_bound(ref, size, live, torch.float32))
    ref, size = O.product(s.dh1, o, None, None, s.w1, n, s.dx2, transposed=True)
    _near(s.dx2[:live], ref[:live], O.product_bound(ref, size, 2 * F, torch.bfloat16)[:live])
    for t in (s.h1, s.a, s.y2, s.da, s.dh1, s.dwgt, s.dx2):  # rows behind the last entry
        assert (t[live:] == -7).all()


def _autograd(s):
    """The layer's function of (x, routing weights, w1, w2) in 64 bits."""
    x, w1, w2 = (v.double().requires_grad_(True) for v in (s.x, s.w1, s.w2))
    wt = s.weights.double().requires_grad_(True)
    y = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in range(E):
        t, k = (s.ids == e).nonzero(as_tuple=True)
        h = x[t] @ w1[e].t()
        a = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:] * wt[t, k][:, None]
        y = y.index_add(0, t, a @ w2[e].t())
    (y * s.dy.double()).sum().backward()
    return y.detach(), x.grad, w1.grad, w2.grad, wt.grad


def test_training_step():
    s = Layer(1)
    s.run()
    torch.cuda.synchronize()
    _check_calls(s)
    y, dx, dw1, dw2, dwt = _autograd(s)
    # Norms: a bf16 rounding is off by 2^-8 of its value at most; y goes through four of them (h1, which the activation
    # passes on at up to 1.1 times in either factor, a, y2 and two sums), a gradient through up to eight.
    for got, ref, roundings in ((s.y, y, 7), (s.dx, dx, 12), (s.dw1, dw1, 12), (s.dw2, dw2, 7)):
        assert (got.double() - ref).norm() <= roundings * 2.0 ** -8 * ref.norm()
    # the routing weights' gradient back at its slots: the entry of (token, slot) through the token's row at its PE
    pe = s.ids.long() // EPR
    rows = torch.full((T, W), -1, dtype=torch.long, device=DEV)
    t, k = (s.buf.sendMap.view(T, K) >= 0).nonzero(as_tuple=True)
    rows[t, pe[t, k]] = s.buf.sendMap.view(T, K)[t, k].long()
    entry = s.of.view(W * M, K)[rows.gather(1, pe)].gather(2, torch.arange(K, device=DEV).expand(T, K)[..., None])[..., 0]
    got = s.dwgt[entry.long()]
    assert (got.double() - dwt).norm() <= 7 * 2.0 ** -8 * dwt.norm()
    dlogits = torch.empty(T, E, device=DEV)
    epdc.epdc_route_grad(s.rcfg, T, s.logits, s.ids, got.contiguous(), dlogits)
    assert torch.isfinite(dlogits).all() and dlogits.abs().max() > 0


def test_training_step_captured_and_on_two_streams():
    s, other = Layer(2), Layer(3)
    s.run(), other.run()
    torch.cuda.synchronize()
    want, want_other = ({k: v.clone() for k, v in l.results().items()} for l in (s, other))
    # captured, replayed with other inputs in between and with eager work and synchronisations
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for i in range(4):
        for t in (s.h1, s.a, s.da, s.dh1, s.y2, s.dx2, s.dw1, s.dw2):
            t.fill_(float("nan") if i % 2 else -7.0)
        s.logits.mul_(-1.0 if i in (1, 2) else 1.0)
        graph.replay()
        torch.cuda.synchronize()
        if i != 1:
            for k, v in s.results().items():
                assert torch.equal(v, want[k]), (i, k)
    # two streams at once
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for l, st in zip((s, other), streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                l.run()
        torch.cuda.synchronize()
        for l, w in ((s, want), (other, want_other)):
            for k, v in l.results().items():
                assert torch.equal(v, w[k]), k


def test_int8_forward():
    """Rows quantised, dispatched as one-byte rows with one scale each, multiplied, activated and quantised in one,
    multiplied; against the formulas on what each call read."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    h, f = 144, 80  # rows of whole 16 bytes
    cfg = epdc.EpCfg(W, h, M, EPR, K, epdc.EPDC_FP8, 1, 1)
    n = W * M * K
    x = _bf(T, h, g=g)
    ids = torch.stack([torch.randperm(E, device=DEV, generator=g)[:K] for _ in range(T)]).to(torch.int32)
    wt = torch.rand(T, K, device=DEV, generator=g)
    w1, w1s = O.int8_rows(torch.randn(E * 2 * f, h, device=DEV, generator=g))
    w2, w2s = O.int8_rows(torch.randn(E * h, f, device=DEV, generator=g))
    w1, w2 = w1.to(DEV).view(E, 2 * f, h), w2.to(DEV).view(E, h, f)
    w1s, w2s = w1s.to(DEV).view(E, 2 * f), w2s.to(DEV).view(E, h)
    q, qs = torch.zeros(T, h, dtype=torch.int8, device=DEV), torch.zeros(T, 1, device=DEV)
    b = epdc.DispatchBuffers(cfg)
    epdc.epdc_int_quantize(1, T, h, BF16, x, None, q, qs)
    epdc.epdc_dispatch(cfg, T, q, ids, wt, qs, b.recvX, b.recvTokIdx, b.recvExpertIds, b.recvWeights, b.recvScales, b.recvCount,
                       b.sendMap, b.scratch)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    row, of = torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(W, M, K, dtype=torch.int32, device=DEV)
    wgt = torch.zeros(n, device=DEV)
    scratch = torch.zeros(epdc.epdc_group_scratch_bytes(cfg, -1) // 4 + 4, dtype=torch.int32, device=DEV)
    epdc.epdc_group_experts(cfg, -1, b.recvExpertIds, b.recvWeights, b.recvCount, off, row, wgt, of, scratch)
    h1 = torch.zeros(n, 2 * f, device=DEV, dtype=torch.bfloat16)
    a, a_s = torch.zeros(n, f, dtype=torch.int8, device=DEV), torch.zeros(n, device=DEV)
    y2 = torch.zeros(n, h, device=DEV)
    epdc.epdc_expert_linear_int(E, 2 * f, h, n, W * M, b.recvX, b.recvScales, off, row, None, w1, w1s, h1, BF16)
    epdc.epdc_expert_gate_int(E, f, n, BF16, h1, off, wgt, a, a_s)
    epdc.epdc_expert_linear_int(E, h, f, n, n, a, a_s, off, None, None, w2, w2s, y2, FP32)
    torch.cuda.synchronize()
    rq, rs = O.int8_rows(x)
    assert torch.equal(q.cpu(), rq) and torch.equal(qs.view(-1).cpu(), rs)
    o = off.tolist()
    live = o[-1]
    ref, _ = O.product(b.recvX.view(torch.int8).view(W * M, h), o, row, None, w1, n, h1, b.recvScales.view(-1), w1s)
    _near(h1[:live], ref[:live], O.int8_bound(ref, torch.bfloat16)[:live])
    rq, rs = O.int8_rows(O.gate(h1[:live], wgt[:live]).float())
    assert torch.equal(a[:live].cpu(), rq) and torch.equal(a_s[:live].cpu(), rs)
    ref, _ = O.product(a, o, None, None, w2, n, y2, a_s, w2s)
    _near(y2[:live], ref[:live], O.int8_bound(ref, torch.float32)[:live])
