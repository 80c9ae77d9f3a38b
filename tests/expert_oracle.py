"""Plain 64-bit implementations (torch, any device) of the experts in bf16 and
int8, from the formulas in include/epdc.h, with the error bounds that the
kernels' roundings allow."""
from __future__ import annotations

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # of a rounding to nearest, relative


def groups_of(offsets, n):
    """[(first, last)] per expert: clamped to [0, n], a group ending at the smallest offset behind its start's."""
    o = [min(max(v, 0), n) for v in offsets]
    out = []
    for e in range(len(o) - 1):
        end = min(o[e + 1:])
        out.append((o[e], max(end, o[e])))
    return out


def _valid(row, n, rows, lo, hi):
    r = torch.arange(lo, hi) if row is None else row[lo:hi].long().cpu()
    return r, (r >= 0) & (r < rows)


def product(x, offsets, entry_row, w, weights, n, out, scales=None, weight_scales=None, transposed=False):
    """out (float64, a copy of what was there) with the groups' rows replaced, and the sum of magnitudes behind
    every element (0 where nothing is written)."""
    out, size = out.double().clone(), torch.zeros(out.shape, dtype=torch.float64, device=out.device)
    for e, (lo, hi) in enumerate(groups_of(offsets, n)):
        if lo >= hi:
            continue
        r, ok = _valid(entry_row, n, x.shape[0], lo, hi)
        b = weights[e].double()
        b = b if transposed else b.t().contiguous()
        a = torch.zeros(hi - lo, b.shape[0], dtype=torch.float64, device=out.device)
        at = ok.nonzero()[:, 0].to(out.device)
        rows = r[ok].to(out.device)
        a[at] = x[rows].double()
        v, s = a @ b, a.abs() @ b.abs()
        if scales is not None:
            f = torch.zeros(hi - lo, 1, dtype=torch.float64, device=out.device)
            f[at, 0] = scales[rows].double()
            f = f * weight_scales[e].double()[None]
            v, s = v * f, v.abs() * f.abs()
        if w is not None:
            v, s = v * w[lo:hi].double()[:, None], s * w[lo:hi].double().abs()[:, None]
        gone = (~ok).to(out.device)
        v[gone] = 0.0
        s[gone] = 0.0
        out[lo:hi], size[lo:hi] = v, s
    return out, size


def weights_grad(d, out_row, x, entry_row, offsets, n, E, base):
    N, H = d.shape[1], x.shape[1]
    v = torch.zeros(E, N, H, dtype=torch.float64, device=d.device)
    s = torch.zeros_like(v)
    for e, (lo, hi) in enumerate(groups_of(offsets, n)):
        r, ok = _valid(entry_row, n, x.shape[0], lo, hi)
        o, ok2 = _valid(out_row, n, d.shape[0], lo, hi)
        ok = ok & ok2
        a, b = d[o[ok].to(d.device)].double().t().contiguous(), x[r[ok].to(d.device)].double()
        v[e], s[e] = a @ b, a.abs() @ b.abs()
    return (v, s) if base is None else (v + base.double(), s + base.double().abs())


def product_bound(ref, size, terms, dtype):
    """terms products summed in fp32, at most a step (2^-23) lost by each addition, one more for the weight or the
    base, then one rounding to dtype."""
    err = (terms + 4) * 2.0 ** -23 * size
    return err + HALF_STEP[dtype] * (ref.abs() + err) + 1e-37


def int8_bound(ref, dtype):
    """The integer sum to fp32, three fp32 products: half a step each; then one rounding."""
    err = 4 * 2.0 ** -24 * (1 + 2.0 ** -20) * ref.abs()
    return err + HALF_STEP[dtype] * (ref.abs() + err) + 1e-37


def gate(h, w):
    g, u = h.double().chunk(2, dim=1)
    a = g * torch.sigmoid(g) * u
    return a if w is None else a * w.double()[:, None]


def gate_bound(h, w, ref, dtype):
    """exp to one step (2 half steps), 1 + t, the quotient, t times it, three products: 9 half steps; a subnormal
    exponential to half of 2^-149."""
    g, u = h.double().chunk(2, dim=1)
    f = 1.0 if w is None else w.double().abs()[:, None]
    err = 9 * 2.0 ** -24 * (1 + 2.0 ** -20) * ref.abs() + 2.0 ** -148 * (g * u).abs() * f
    return err + HALF_STEP[dtype] * (ref.abs() + err) + 1e-37


def gate_grad(h, w, d):
    """dH, dw and the magnitudes behind them."""
    g, u = h.double().chunk(2, dim=1)
    d = d.double()
    s, rest = torch.sigmoid(g), torch.sigmoid(-g)
    dw = (d * g * s * u).sum(1)
    size_w = (d * g * s * u).abs().sum(1)
    e = d if w is None else d * w.double()[:, None]
    dh = torch.cat([e * u * s * (1 + g * rest), e * g * s], dim=1)
    size = torch.cat([(e * u).abs() * s * (1 + g.abs() * rest), (e * g).abs() * s], dim=1)
    return dh, dw, size, size_w


def gate_grad_bounds(h, dh, dw, size, size_w, dtype):
    """As gate_bound, with 1 + g rest (two more roundings of the exponential's kind: 6 half steps), three products;
    the row's sum adds a half step per term."""
    cols = h.shape[1] // 2
    err = 16 * 2.0 ** -24 * size
    return (err + HALF_STEP[dtype] * (dh.abs() + err) + 1e-36, (cols + 16) * 2.0 ** -24 * size_w + 1e-36)


def int8_rows(x):
    """Codes and scales of rows of fp32 values: both quotients in fp32, rounded to nearest even (IEEE division)."""
    x = x.float().cpu()
    most = x.abs().amax(1)
    bad = ~torch.isfinite(x).all(1)
    scale = torch.where(bad, float("nan"), most / 127.0)
    q = torch.round(x / scale[:, None]).clamp(-127, 127)
    q = torch.where((scale > 0)[:, None], q, 0.0)
    return q.to(torch.int8), scale.float()
