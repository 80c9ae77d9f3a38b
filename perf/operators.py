"""The operators next to dispatch and combine, as cases to measure: routing and
its gradient, microscaled fp4 quantisation, grouping of received rows by
expert, and the experts' product over the groups.

A case is a plain dict; ``prepare`` makes its inputs on the GPU, ``run`` is
one pass (plain torch operations, or the library's calls where ``own`` is
set), ``exact`` the same result from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

INF = math.inf
FLOAT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    route = dict(op="route", experts=256, topk=8, dtype="bf16", score="sigmoid", bias=True, groups=8, keep=4,
                 group_top=2, renorm=True, scale=2.5, masked=0.0, padded=0.0)
    grad = dict(op="route_grad", experts=256, topk=8, dtype="fp32", score="softmax", renorm=False, scale=1.0,
                dropped=0.0, padded=0.0)
    return [
        # one decode step: a few sequences' tokens, group-limited sigmoid routing with a balance bias
        dict(route, name="route_decode_t8", tokens=8),
        # prefill of one rank, softmax over 256 experts, fp32 logits, renormalised top-8
        dict(route, name="route_softmax_t4096", tokens=4096, dtype="fp32", score="softmax", bias=False, groups=1,
             keep=1, group_top=1, scale=1.0),
        # a large training batch in one call, ragged: padding rows with no expert left, some experts masked out
        dict(route, name="route_groups_t65521", tokens=65521, masked=0.02, padded=0.03),
        # training, 512 tokens of top-6 over 128 experts, softmax without renormalisation: the dense gradient
        dict(grad, name="route_grad_t512", tokens=512, experts=128, topk=6, dtype="bf16"),
        # training, a large batch, renormalised sigmoid weights: a sparse gradient into a dense tensor
        dict(grad, name="route_grad_t65536", tokens=65536, score="sigmoid", renorm=True, scale=2.5, dropped=0.05),
        # the wire's round trip for 128 tokens: quantised for the dispatch, read back as bf16
        dict(op="mx", name="mx_t128_h7168", tokens=128, cols=7168, dtype="bf16", out="bf16"),
        # the same for 16384 tokens
        dict(op="mx", name="mx_t16384_h7168", tokens=16384, cols=7168, dtype="bf16", out="bf16"),
        # received rows of 8 windows of at most 128 rows, 8 experts a rank, all ranks' experts
        dict(op="group", name="group_w8_m128", windows=8, rows=128, experts=8, topk=8, rank=-1, fill=0.6, skew=0.0),
        # one rank's view: 8 sources of up to 4096 rows, 32 experts of its own, popular and rare ones
        dict(op="group", name="group_w8_m4096", windows=8, rows=4096, experts=32, topk=8, rank=3, fill=0.4, skew=1.1),
        # decode: 8 tokens' rows over one rank's 32 experts, first product of an expert (h7168 -> 4096)
        dict(op="product", name="product_decode_64", experts=32, entries=64, rows=8, cols=4096, hidden=7168,
             out="bf16", gather=True, weighted=False, skew=0.0),
        # second product of an expert over sorted rows, weighted, uneven groups, fp32 sums for the combine
        dict(op="product", name="product_ragged_2047", experts=32, entries=2047, rows=2047, cols=7168, hidden=2048,
             out="fp32", gather=False, weighted=True, skew=1.1),
        # prefill: one rank's rows of 8 sources, first product of an expert
        dict(op="product", name="product_prefill_32768", experts=32, entries=32768, rows=16384, cols=4096,
             hidden=7168, out="bf16", gather=True, weighted=False, skew=0.4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "mx", "group", "product"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        each = rng.randint(2, 512 // groups)
        experts = groups * each
        keep = rng.randint(1, groups)
        case = dict(op=op, experts=experts, topk=rng.randint(1, min(16, keep * each)), dtype=rng.choice(["bf16", "fp32"]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5, 16.0]),
                    tokens=max(1, min(_log(rng, 1, 60000), (12 << 20) // experts)), padded=rng.choice([0.0, 0.1]))
        if op == "route":
            return dict(case, bias=rng.random() < 0.6, groups=groups, keep=keep, group_top=rng.randint(1, min(2, each)),
                        masked=rng.choice([0.0, 0.05, 0.5]))
        return dict(case, dropped=rng.choice([0.0, 0.1]))
    if op == "mx":
        cols = 32 * _log(rng, 1, 400)
        return dict(op=op, tokens=max(1, min(_log(rng, 1, 40000), (100 << 20) // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "fp32"]), out=rng.choice(["bf16", "fp32"]))
    if op == "group":
        windows = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, windows=windows, rows=_log(rng, 40, 30000 // windows), experts=_log(rng, 1, 64),
                    topk=rng.randint(1, 8), rank=rng.choice([-1, 0, windows - 1]), fill=rng.uniform(0.2, 1.0),
                    skew=rng.choice([0.0, 1.1]))
    hidden, cols = 32 * _log(rng, 1, 128), 8 * _log(rng, 1, 512)
    entries = _log(rng, 1, 16000)
    return dict(op=op, experts=_log(rng, 1, 48), entries=entries, rows=max(1, entries // rng.choice([1, 2, 8])),
                cols=cols, hidden=hidden, out=rng.choice(["bf16", "fp32"]), gather=rng.random() < 0.7,
                weighted=rng.random() < 0.5, skew=rng.choice([0.0, 0.4, 1.1]))


# ---- inputs -------------------------------------------------------------------------------------------------------


def _popularity(n, skew):
    p = torch.arange(1, n + 1, dtype=torch.float32, device="cuda") ** -skew
    return p / p.sum()


def _routing_inputs(c, g):
    """Router logits: a spread of popular and rare experts under per-token noise, in the case's type."""
    T, E = c["tokens"], c["experts"]
    l = torch.randn(T, E, device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g)
    l = l.to(FLOAT[c["dtype"]])
    pad = torch.rand(T, device="cuda", generator=g) < c["padded"]
    return l, pad


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    st = {"case": c}
    op = c["op"]
    dev = "cuda"
    if op == "route":
        l, pad = _routing_inputs(c, g)
        if c["masked"]:
            l.masked_fill_(torch.rand(l.shape, device=dev, generator=g) < c["masked"], -INF)
        l[pad] = -INF
        st["logits"] = l
        st["bias"] = 0.1 * torch.randn(c["experts"], device=dev, generator=g) if c["bias"] else None
        st["ids"] = torch.empty(c["tokens"], c["topk"], dtype=torch.int32, device=dev)
        st["weights"] = torch.empty(c["tokens"], c["topk"], dtype=torch.float32, device=dev)
    elif op == "route_grad":
        l, pad = _routing_inputs(c, g)
        ids = torch.topk(l.float(), c["topk"], dim=1).indices.to(torch.int32)
        ids[torch.rand(ids.shape, device=dev, generator=g) < c["dropped"]] = -1
        ids[pad] = -1
        st["logits"], st["ids"] = l, ids.contiguous()
        st["dw"] = torch.randn(ids.shape, device=dev, generator=g)
        st["dlogits"] = torch.empty_like(l)
    elif op == "mx":
        x = torch.randn(c["tokens"], c["cols"], device=dev, generator=g)
        x *= 1.0 + 20.0 * (torch.rand(c["cols"], device=dev, generator=g) < 0.01)  # a few outlier channels
        x *= torch.exp(0.5 * torch.randn(c["tokens"], 1, device=dev, generator=g))
        st["x"] = x.to(FLOAT[c["dtype"]])
        st["q"] = torch.empty(c["tokens"], c["cols"] // 2, dtype=torch.uint8, device=dev)
        st["scales"] = torch.empty(c["tokens"], (c["cols"] + 127) // 128, dtype=torch.int32, device=dev)
        st["out"] = torch.empty(c["tokens"], c["cols"], dtype=FLOAT[c["out"]], device=dev)
    elif op == "group":
        W, M, K, epr = c["windows"], c["rows"], c["topk"], c["experts"]
        E = W * epr
        K = c["topk"] = min(K, E)
        # distinct experts of a token by the largest of log popularity + Gumbel noise
        u = torch.rand(W * M, E, device=dev, generator=g).clamp_min_(1e-9)
        u = _popularity(E, c["skew"])[torch.randperm(E, device=dev, generator=g)].log() - torch.log(-torch.log(u))
        ids = torch.topk(u, K, dim=1).indices.to(torch.int32)
        del u
        ids[torch.rand(ids.shape, device=dev, generator=g) < 0.02] = -1  # dropped slots
        count = torch.rand(W, device=dev, generator=g) * 0.5 + 0.75
        st["count"] = (count * c["fill"] * M).round().clamp(0, M).to(torch.int32)
        st["ids"] = ids.view(W, M, K).contiguous()
        st["w"] = torch.rand(W, M, K, device=dev, generator=g)
        groups = E if c["rank"] < 0 else epr
        st["offsets"] = torch.zeros(groups + 1, dtype=torch.int32, device=dev)
        st["entry_row"] = torch.full((W * M * K,), -1, dtype=torch.int32, device=dev)
        st["entry_weight"] = torch.zeros(W * M * K, device=dev)
        st["entry_of"] = torch.full((W, M, K), -1, dtype=torch.int32, device=dev)
    else:
        E, n, R, N, H = c["experts"], c["entries"], c["rows"], c["cols"], c["hidden"]
        if not c["gather"]:
            R = c["rows"] = n
        e = torch.multinomial(_popularity(E, c["skew"])[torch.randperm(E, device=dev, generator=g)], n, True, generator=g)
        row = torch.randint(R, (n,), device=dev, generator=g)
        order = torch.argsort(e * R + row, stable=True)
        counts = torch.bincount(e, minlength=E)
        st["most"] = int(counts.max())  # the plain form pads every group to this
        st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), counts.cumsum(0)]).to(torch.int32)
        st["entry_row"] = row[order].to(torch.int32) if c["gather"] else None
        st["entry_weight"] = torch.rand(n, device=dev, generator=g) if c["weighted"] else None
        x = torch.randn(R, H, device=dev, generator=g)
        st["a"], st["as"] = _to_mx(x)
        del x
        st["b"] = torch.empty(E, N, H // 2, dtype=torch.uint8, device=dev)
        st["bs"] = torch.empty(E, N, (H + 127) // 128, dtype=torch.int32, device=dev)
        for i in range(E):
            st["b"][i], st["bs"][i] = _to_mx(0.02 * torch.randn(N, H, device=dev, generator=g))
        st["out"] = torch.zeros(n, N, dtype=FLOAT[c["out"]], device=dev)
    return st


# ---- the plain forms ----------------------------------------------------------------------------------------------


def _route(c, logits, bias):
    # 64 bits: which of two nearly equal scores is larger decides an expert
    T, E, G, K = c["tokens"], c["experts"], c["groups"], c["topk"]
    l = logits.double()
    none = torch.isnan(l) | (l == -INF)
    if c["score"] == "softmax":
        top = l.masked_fill(none, -INF).amax(1, keepdim=True)
        e = torch.where(none, 0.0, torch.where(l == top, 1.0, torch.exp(l - top)))
        s = e / e.sum(1, keepdim=True).clamp_min(1.0)
    else:
        s = torch.where(none, 0.0, 1.0 / (1.0 + torch.exp(-l)))
    choice = s if bias is None else s + bias.double()
    choice = choice.masked_fill(none | torch.isnan(choice), -INF)
    key = l.masked_fill(none, -INF) if bias is None else choice
    if c["keep"] < G:
        if c["group_top"] == 1:
            best = key.view(T, G, E // G).amax(2)
        else:
            best = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values[:, :, :2]
            best = torch.where(best[:, :, :1] == -INF, -INF, best.masked_fill(best == -INF, 0.0)).sum(2)
        first = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, first, True)
        key = key.masked_fill(~kept.repeat_interleave(E // G, dim=1), -INF)
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)
    key, ids = key[:, :K], ids[:, :K]
    w = s.gather(1, ids).masked_fill(key == -INF, 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids.masked_fill(key == -INF, -1).to(torch.int32), (w * c["scale"]).float()


def _route_grad(c, logits, ids, dw):
    l = logits.float()
    ok = ids >= 0
    at = ids.clamp_min(0).long()
    g = torch.where(ok, dw, 0.0) * c["scale"]
    sel = l.gather(1, at).masked_fill(~ok, -INF)
    if c["score"] == "softmax" and not c["renorm"]:
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        dot = (g * p.gather(1, at)).sum(1, keepdim=True)
        return (p * (torch.zeros_like(l).scatter_add_(1, at, g) - dot)).to(logits.dtype)
    if c["score"] == "softmax":
        e = torch.where(ok, torch.exp(sel - sel.amax(1, keepdim=True)), 0.0)
        r, q = e / e.sum(1, keepdim=True).clamp_min(1.0), 1.0
    else:
        r, q = torch.where(ok, torch.sigmoid(sel), 0.0), torch.sigmoid(-sel)
        if c["renorm"]:
            total = r.sum(1, keepdim=True)
            r = torch.where(total > 0, r / total, 0.0)
    d = torch.where(ok, r * q * (g - ((g * r).sum(1, keepdim=True) if c["renorm"] else 0.0)), 0.0)
    return torch.zeros_like(l).scatter_add_(1, at, d).to(logits.dtype)


def _to_mx(x):
    """Rows of 32-element blocks as e2m1 codes (two a byte, the first low) and their power-of-two scales (four
    bytes a 32-bit word, filled up with 127)."""
    rows, cols = x.shape
    v = x.float().view(rows, cols // 32, 32)
    most = v.abs().amax(2)
    byte = torch.where(most > 0, torch.frexp(most).exponent + 124, 0).clamp(0, 254)
    byte = torch.where(torch.isfinite(most), byte, 255)
    a = v.abs() * torch.exp2(127.0 - byte.double()).float()[..., None]
    # ties go to the even code
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code |= torch.signbit(v).to(torch.uint8) << 3
    code = torch.where((byte == 255)[..., None], 0, code).view(rows, cols // 2, 2)
    words = torch.full((rows, (cols + 127) // 128 * 4), 127, dtype=torch.uint8, device=x.device)
    words[:, :cols // 32] = byte.to(torch.uint8)
    return code[..., 0] | code[..., 1] << 4, words.view(torch.int32)


def _from_mx(q, words, cols):
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    values = torch.cat([values, -values])
    pairs = torch.stack([values.repeat(16), values.repeat_interleave(16)], dim=1)  # by byte: low code, high code
    byte = words.contiguous().view(torch.uint8)[..., :cols // 32]
    scale = torch.where(byte == 255, math.nan, torch.exp2(byte.double() - 127.0)).float()
    v = pairs[q.int()].view(*q.shape[:-1], cols // 32, 32)
    return (v * scale[..., None]).view(*q.shape[:-1], cols)


def _group(c, ids, w, count):
    W, M, K = ids.shape
    epr, rank = c["experts"], c["rank"]
    base = torch.arange(W, device=ids.device) * epr if rank < 0 else torch.full((W,), rank * epr, device=ids.device)
    rel = ids - base[:, None, None]
    ok = (rel >= 0) & (rel < epr) & (torch.arange(M, device=ids.device)[None, :, None] < count[:, None, None])
    groups = W * epr if rank < 0 else epr
    group = torch.where(ok, ids - (0 if rank < 0 else rank * epr), groups).view(-1).long()
    order = torch.sort(group, stable=True).indices
    at = torch.arange(W * M * K, device=ids.device)
    n = ok.sum()
    sizes = torch.zeros(groups + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, group, torch.ones_like(group))
    offsets = torch.cat([sizes.new_zeros(1), sizes[:groups].cumsum(0)])
    of = torch.empty_like(at).scatter_(0, order, at)
    return {"offsets": offsets.to(torch.int32), "entry_row": torch.where(at < n, order // K, -1).to(torch.int32),
            "entry_weight": torch.where(at < n, w.reshape(-1)[order], 0.0),
            "entry_of": torch.where(of < n, of, -1).to(torch.int32).view(W, M, K)}


def _product(c, st):
    E, n, N, H, most = c["experts"], c["entries"], c["cols"], c["hidden"], st["most"]
    a = _from_mx(st["a"], st["as"], H)
    b = _from_mx(st["b"], st["bs"], H).transpose(1, 2).contiguous()
    at = st["offsets"][:-1, None] + torch.arange(most, device=a.device)  # every group padded to the largest
    ok = at < st["offsets"][1:, None]
    at = at.clamp_max(n - 1).long()
    row = at if st["entry_row"] is None else st["entry_row"][at].long()
    v = torch.bmm(torch.where(ok[..., None], a[row], 0.0), b)
    if st["entry_weight"] is not None:
        v = v * st["entry_weight"][at][..., None]
    at = torch.where(ok, at, n).view(-1)  # the padding goes to a row of its own
    return torch.empty(n + 1, N, dtype=FLOAT[c["out"]], device=a.device).index_copy_(0, at, v.to(FLOAT[c["out"]]).view(-1, N))[:n]


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "route":
        return dict(zip(("ids", "weights"), _route(c, st["logits"], st["bias"])))
    if op == "route_grad":
        return {"dlogits": _route_grad(c, st["logits"], st["ids"], st["dw"])}
    if op == "mx":
        q, words = _to_mx(st["x"])
        return {"out": _from_mx(q, words, c["cols"]).to(FLOAT[c["out"]])}
    if op == "group":
        return _group(c, st["ids"], st["w"], st["count"])
    return {"out": _product(c, st)}


# ---- the library's calls ------------------------------------------------------------------------------------------


def _calls(st):
    """The calls of one pass, their arguments marshalled once for the state's fixed buffers, as a serving or training
    loop keeps them."""
    import combine_count_amd as epdc
    c = st["case"]
    op = c["op"]
    kind = {"bf16": epdc.EPDC_BF16, "fp32": epdc.EPDC_FP32}
    if op in ("route", "route_grad"):
        cfg = epdc.RouteCfg(numExperts=c["experts"], numExpertPerToken=c["topk"], dtype=kind[c["dtype"]],
                            score={"softmax": epdc.EPDC_SOFTMAX, "sigmoid": epdc.EPDC_SIGMOID}[c["score"]],
                            numGroups=c.get("groups", 1), groupsPerToken=c.get("keep", 1), groupTop=c.get("group_top", 1),
                            renormalize=int(c["renorm"]), routedScale=c["scale"])
        if op == "route":
            return [epdc.prepare_route(cfg, c["tokens"], st["logits"], st["bias"], st["ids"], st["weights"])]
        return [epdc.prepare_route_grad(cfg, c["tokens"], st["logits"], st["ids"], st["dw"], st["dlogits"])]
    if op == "mx":
        return [epdc.prepare_mx_quantize(1, c["tokens"], c["cols"], kind[c["dtype"]], st["x"], None, st["q"], st["scales"]),
                epdc.prepare_mx_dequantize(1, c["tokens"], c["cols"], st["q"], st["scales"], None, st["out"], kind[c["out"]])]
    if op == "group":
        cfg = epdc.EpCfg(c["windows"], 1024, c["rows"], c["experts"], c["topk"], epdc.EPDC_BF16, 1, 0)
        scratch = torch.zeros(epdc.epdc_group_scratch_bytes(cfg, c["rank"]) // 4, dtype=torch.int32, device="cuda")
        return [epdc.prepare_group_experts(cfg, c["rank"], st["ids"], st["w"], st["count"], st["offsets"], st["entry_row"],
                                           st["entry_weight"], st["entry_of"], scratch)]
    return [epdc.prepare_expert_product(c["experts"], c["cols"], c["hidden"], c["entries"], c["rows"], st["a"], st["as"],
                                        st["offsets"], st["entry_row"], st["entry_weight"], st["b"], st["bs"], st["out"],
                                        kind[c["out"]])]


RESULTS = {"route": ("ids", "weights"), "route_grad": ("dlogits",), "mx": ("out",),
           "group": ("offsets", "entry_row", "entry_weight", "entry_of"), "product": ("out",)}


def run(st):
    if not own:
        return _plain(st)
    if "calls" not in st:
        st["calls"] = _calls(st)
    for call in st["calls"]:
        call()
    return {k: st[k] for k in RESULTS[st["case"]["op"]]}


# ---- what a pass cannot do without --------------------------------------------------------------------------------


def work(case):
    c = case
    op = c["op"]
    if op == "route":
        T, E = c["tokens"], c["experts"]
        return {"bytes": T * E * SIZE[c["dtype"]] + (E * 4 if c["bias"] else 0) + T * c["topk"] * 8, "flops": 8 * T * E}
    if op == "route_grad":
        T, E, K = c["tokens"], c["experts"], c["topk"]
        dense = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": T * (E + (E if dense else K)) * SIZE[c["dtype"]] + T * K * 8, "flops": T * (8 * E if dense else 12 * K)}
    if op == "mx":  # x in, codes and scales out and in, values out
        n = c["tokens"] * c["cols"]
        return {"bytes": n * (SIZE[c["dtype"]] + SIZE[c["out"]]) + 2 * (n // 2 + n // 32), "flops": 4 * n}
    if op == "group":
        E = c["windows"] * c["experts"]
        R, K = c["windows"] * c["rows"] * min(1.0, c["fill"]), min(c["topk"], E)
        n = R * K / c["windows"]  # every window holds its own rank's share, or a rank its own
        return {"bytes": R * K * 4 + c["windows"] * c["rows"] * K * 4 + n * 12, "flops": R * K}
    E, n, N, H = c["experts"], c["entries"], c["cols"], c["hidden"]
    touched = E * (1.0 - (1.0 - 1.0 / E) ** n)
    R = min(n, c["rows"]) if c["gather"] else n
    return {"bytes": (touched * N + R) * (H // 2 + H // 32) + n * N * SIZE[c["out"]], "flops": 2 * n * N * H}


# ---- 64 bits, from the definitions --------------------------------------------------------------------------------


def _exact_route(c, st):
    T, E, G = c["tokens"], c["experts"], c["groups"]
    l = st["logits"].double().cpu().numpy()
    b = None if st["bias"] is None else st["bias"].double().cpu().numpy()
    out = np.zeros((T, c["topk"]))
    step = max(1, (1 << 22) // E)
    for t in range(0, T, step):
        x = np.where(np.isnan(l[t:t + step]), -INF, l[t:t + step])
        dead = x == -INF
        with np.errstate(all="ignore"):
            if c["score"] == "softmax":
                p = np.where(dead, 0.0, np.exp(x - np.where(dead.all(1), 0.0, x.max(1))[:, None]))
                p /= np.maximum(p.sum(1, keepdims=True), 1.0)
            else:
                p = np.where(dead, 0.0, 1.0 / (1.0 + np.exp(-x)))
        v = p if b is None else p + b
        v = np.where(dead, -INF, v)
        k = x if b is None else v
        if c["keep"] < G:
            u = (k if c["group_top"] == 1 else v).reshape(len(x), G, E // G)
            u = -np.partition(-u, c["group_top"] - 1, axis=2)[:, :, :c["group_top"]]
            u = np.where((u == -INF).all(2), -INF, np.where(u == -INF, 0.0, u).sum(2))
            off = np.argsort(-u, axis=1, kind="stable")[:, c["keep"]:]
            gone = np.zeros((len(x), G), dtype=bool)
            np.put_along_axis(gone, off, True, 1)
            k = np.where(np.repeat(gone, E // G, axis=1), -INF, k)
        at = np.argsort(-k, axis=1, kind="stable")[:, :c["topk"]]
        w = np.where(np.take_along_axis(k, at, 1) == -INF, 0.0, np.take_along_axis(p, at, 1))
        if c["renorm"]:
            w = w / np.where(w.sum(1) > 0, w.sum(1), 1.0)[:, None]
        out[t:t + step] = w * c["scale"]
    return {"ids": None, "weights": torch.from_numpy(out)}  # whole numbers have to be equal: no value in 64 bits


def _exact_route_grad(c, st):
    """By automatic differentiation of the weights in 64 bits."""
    l = st["logits"].double().requires_grad_(True)
    ids, ok = st["ids"].clamp_min(0).long(), st["ids"] >= 0
    if c["score"] == "softmax":
        s = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    w = s.gather(1, ids) * ok
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + (~ok).all(1, keepdim=True))
    (w * st["dw"].double() * c["scale"]).sum().backward()
    return {"dlogits": l.grad}


def _exact_mx(c, st):
    """Every element to the nearest of the sixteen values, of two equally near ones to that with an even code."""
    x = st["x"].double().view(c["tokens"], -1, 32)
    most = x.abs().amax(2, keepdim=True)
    unit = torch.exp2((torch.floor(torch.log2(most.clamp_min(1e-300))) - 2.0).clamp(-127.0, 127.0))
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    a = x.abs() / unit
    best, far = torch.zeros_like(a), a.clone()
    for code, value in enumerate(grid):
        d = (a - value).abs()
        take = (d < far) | ((d == far) & (code % 2 == 0))
        best, far = torch.where(take, value, best), torch.where(take, d, far)
    return {"out": (torch.copysign(best, x) * unit).view(c["tokens"], c["cols"])}


def _exact_product(c, st):
    H = c["hidden"]
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    value = torch.tensor(grid + [-v for v in grid], dtype=torch.float64, device="cuda")

    def dense(q, words):
        both = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2)
        unit = torch.pow(2.0, words.contiguous().view(torch.uint8)[:, :H // 32].double() - 127.0)
        return value[both.int()] * unit.repeat_interleave(32, dim=1)

    a, bounds = dense(st["a"], st["as"]), st["offsets"].tolist()
    out = torch.zeros(c["entries"], c["cols"], dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo < hi:
            rows = a[lo:hi] if st["entry_row"] is None else a[st["entry_row"][lo:hi].long()]
            out[lo:hi] = rows @ dense(st["b"][e], st["bs"][e]).t().contiguous()
    return {"out": out if st["entry_weight"] is None else out * st["entry_weight"].double()[:, None]}


def _exact_group(c, st):
    ids, count, rank, epr = st["ids"].cpu().numpy(), st["count"].cpu().numpy(), c["rank"], c["experts"]
    p, r, k = np.nonzero((ids >= 0) & (np.arange(c["rows"])[None, :, None] < count[:, None, None]))
    e = ids[p, r, k]
    mine = e // epr == (p if rank < 0 else rank)
    p, r, k, e = p[mine], r[mine], k[mine], e[mine]
    order = np.lexsort((k, r, p, e))
    w = np.zeros(ids.size)
    w[:len(e)] = st["w"].cpu().numpy()[p[order], r[order], k[order]]
    return {"offsets": None, "entry_row": None, "entry_weight": torch.from_numpy(w), "entry_of": None}  # whole numbers: None


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    of = {"route": _exact_route, "route_grad": _exact_route_grad, "mx": _exact_mx, "group": _exact_group, "product": _exact_product}
    return of[c["op"]](c, st)
