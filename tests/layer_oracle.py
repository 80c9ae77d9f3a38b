"""Plain 64-bit implementations (numpy, on the host) of the operators next to
dispatch and combine, from the formulas in include/epdc.h: routing and its
gradient, fp4x2 quantisation, grouping by expert, the experts' product."""
from __future__ import annotations

import numpy as np

INF = np.inf
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scores(l, softmax):
    """[T][E] float64 scores, 0 for a masked logit."""
    l = np.asarray(l, dtype=np.float64)
    dead = np.isnan(l) | (l == -INF)
    x = np.where(dead, -INF, l)
    with np.errstate(all="ignore"):
        if softmax:
            top = np.max(x, axis=1, keepdims=True)
            e = np.where(dead, 0.0, np.where(x == top, 1.0, np.exp(x - top)))
            return e / np.maximum(e.sum(1, keepdims=True), 1.0)
        return np.where(dead, 0.0, 1.0 / (1.0 + np.exp(-x)))


def route(l, bias, K, softmax, G=1, keep=1, top=1, renorm=False, scale=1.0):
    l = np.asarray(l, dtype=np.float64)
    T, E = l.shape
    s = scores(l, softmax)
    dead = np.isnan(l) | (l == -INF)
    with np.errstate(invalid="ignore"):
        c = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    dead = dead | np.isnan(c) | (c == -INF)
    ids = np.full((T, K), -1, dtype=np.int32)
    w = np.zeros((T, K))
    per = E // G
    for t in range(T):
        key = {e: (l[t, e] if bias is None else c[t, e]) for e in range(E) if not dead[t, e]}
        if keep < G:
            score = {}
            for g in range(G):
                members = [e for e in range(g * per, (g + 1) * per) if e in key]
                if not members:
                    continue
                if top == 1:
                    score[g] = max(key[e] for e in members)
                else:
                    score[g] = sum(sorted((c[t, e] for e in members), reverse=True)[:2])
            best = sorted(score, key=lambda g: (-score[g], g))[:keep]
            key = {e: v for e, v in key.items() if e // per in best}
        chosen = sorted(key, key=lambda e: (-key[e], e))[:K]
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = s[t, chosen]
    if renorm:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return ids, w * scale


def weights_of(l, ids, softmax, renorm, scale):
    """The K weights as a function of the logits, the chosen experts fixed."""
    s = scores(l, softmax)
    E = s.shape[1]
    ok = (ids >= 0) & (ids < E)
    w = np.where(ok, np.take_along_axis(s, np.where(ok, ids, 0), 1), 0.0)
    if renorm:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return w * scale


def route_grad(l, ids, dw, softmax, renorm, scale):
    """(gradient, magnitude of what is summed in it) in 64 bits."""
    l = np.asarray(l, dtype=np.float64)
    T, E = l.shape
    s = scores(l, softmax)
    ok = (ids >= 0) & (ids < E)
    at = np.where(ok, ids, 0)
    live = np.take_along_axis(~(np.isnan(l) | (l == -INF)), at, 1)
    ok = ok & live
    g = np.where(ok, np.asarray(dw, dtype=np.float64), 0.0) * scale
    sel = np.where(ok, np.take_along_axis(s, at, 1), 0.0)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    rows = np.arange(T)[:, None]
    if softmax and not renorm:
        dense, dmag = np.zeros((T, E)), np.zeros((T, E))
        np.add.at(dense, (rows, at), g)
        np.add.at(dmag, (rows, at), np.abs(g))
        out = s * (dense - (g * sel).sum(1, keepdims=True))
        mag = s * (dmag + (np.abs(g) * sel).sum(1, keepdims=True))
        return out, mag
    with np.errstate(all="ignore"):
        if softmax:  # over the chosen alone, so that a small share of the token's mass keeps its precision
            x = np.where(ok, np.take_along_axis(l, at, 1), -INF)
            m = x.max(1, keepdims=True)
            sel = np.where(ok, np.where(x == m, 1.0, np.exp(x - m)), 0.0)
            q = np.ones_like(sel)
        else:
            q = np.where(ok, 1.0 / (1.0 + np.exp(np.take_along_axis(l, at, 1))), 0.0)
    r, dot, dmag = sel, 0.0, 0.0
    if renorm:
        total = sel.sum(1, keepdims=True)
        r = np.where(total > 0, sel / np.where(total > 0, total, 1.0), 0.0)
        dot, dmag = (g * r).sum(1, keepdims=True), (np.abs(g) * r).sum(1, keepdims=True)
    np.add.at(out, (rows, at), np.where(ok, r * q * (g - dot), 0.0))
    np.add.at(mag, (rows, at), np.where(ok, r * q * (np.abs(g) + dmag), 0.0))
    return out, mag


def mx_quantize(x):
    """x [R][C] float64 -> codes [R][C] uint8 (0..15) and scale bytes [R][C/32] uint8."""
    R, C = x.shape
    v = np.asarray(x, dtype=np.float64).reshape(R, C // 32, 32)
    finite = np.isfinite(v).all(2)
    m = np.where(finite, np.abs(np.where(np.isfinite(v), v, 0.0)).max(2), 0.0)
    e = np.frexp(m)[1] - 1  # floor(log2 m)
    byte = np.where(m > 0, np.clip(e + 125, 0, 254), 0)
    byte = np.where(finite, byte, 255)
    a = np.where(finite[..., None], np.abs(np.where(np.isfinite(v), v, 0.0)), 0.0) * np.exp2(127.0 - byte)[..., None]
    # nearest of the grid; of two equally near ones that with the even code
    d = np.abs(a[..., None] - GRID)
    near = d == d.min(-1, keepdims=True)
    code = np.where(near & (np.arange(8) % 2 == 0), 1, 0)
    code = np.where(code.any(-1), code.argmax(-1), near.argmax(-1)).astype(np.uint8)
    code |= (np.signbit(v) & finite[..., None]).astype(np.uint8) << 3
    return code.reshape(R, C), byte.astype(np.uint8)


def pack(codes, byte):
    """Codes and scale bytes as the device arrays hold them: q [R][C/2], words [R][S] int32."""
    R, C = codes.shape
    q = codes[:, 0::2] | codes[:, 1::2] << 4
    words = np.full((R, (C + 127) // 128 * 4), 127, dtype=np.uint8)
    words[:, :C // 32] = byte
    return np.ascontiguousarray(q), words.view(np.int32)


def unpack(q, words):
    C = q.shape[1] * 2
    codes = np.empty((q.shape[0], C), dtype=np.uint8)
    codes[:, 0::2], codes[:, 1::2] = q & 15, q >> 4
    return codes, np.ascontiguousarray(words).view(np.uint8).reshape(q.shape[0], -1)[:, :C // 32]


def mx_values(codes, byte):
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    unit = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127.0))
    R, C = codes.shape
    return (v.reshape(R, C // 32, 32) * unit[..., None]).reshape(R, C)


def group(ids, count, epr, rank):
    """offsets, entry rows, entry slots' flat indices and entryOf."""
    W, M, K = ids.shape
    groups = (W if rank < 0 else 1) * epr
    lists = [[] for _ in range(groups)]
    for w in range(W):
        first = (w if rank < 0 else rank) * epr
        for r in range(min(max(int(count[w]), 0), M)):
            for k in range(K):
                e = int(ids[w, r, k])
                if first <= e < first + epr:
                    lists[e - (0 if rank < 0 else first)].append((w * M + r) * K + k)
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in lists])]).astype(np.int32)
    slots = np.array([s for v in lists for s in v], dtype=np.int64)
    of = np.full(W * M * K, -1, dtype=np.int32)
    of[slots] = np.arange(len(slots))
    return offsets, (slots // K).astype(np.int32), slots, of.reshape(W, M, K)


def product(a, b, offsets, rows, weight, n):
    """(out, sum of |products|) [n][N] for a [R][H], b [E][N][H] values; entries outside the groups: NaN."""
    N = b.shape[1]
    out, mag = np.full((n, N), np.nan), np.zeros((n, N))
    E = b.shape[0]
    for e in range(E):
        lo = min(max(int(offsets[e]), 0), n)
        hi = min(max(int(min(offsets[e + 1:])), lo), n)  # the smallest offset behind the group's start
        if lo == hi:
            continue
        r = np.arange(lo, hi) if rows is None else rows[lo:hi]
        ok = (r >= 0) & (r < a.shape[0])
        x = np.where(ok[:, None], a[np.where(ok, r, 0)], 0.0)
        out[lo:hi], mag[lo:hi] = x @ b[e].T, np.abs(x) @ np.abs(b[e]).T
        if weight is not None:
            w = weight[lo:hi].astype(np.float64)[:, None]
            out[lo:hi] *= w
            mag[lo:hi] *= np.abs(w)
    return out, mag
