"""The experts in bf16 and int8, as cases to measure: the products grouped by
expert with their gradients, the gated activation between them with its
gradient, and the int8 form with scales per token and channel.

A case is a plain dict; ``prepare`` makes its inputs on the GPU, ``run`` is
one pass (plain torch operations, or the library's calls where ``own`` is
set), ``exact`` the same result from the definition in 64 bits.
"""
import math

import torch

own = False

FLOAT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    product = dict(op="product", experts=32, cols=4096, hidden=7168, out="bf16", gather=True, weighted=False, skew=0.0)
    return [
        # decode: 8 tokens' rows over one rank's 32 experts, first product of an expert, gate and up columns side by side
        dict(product, name="product_decode_64", entries=64, rows=8),
        # second product of an expert over sorted rows, weighted, uneven groups, fp32 sums for the combine
        dict(product, name="product_ragged_2047", entries=2047, rows=2047, cols=7168, hidden=2048, out="fp32", gather=False,
             weighted=True, skew=1.1),
        # prefill, or a training step's forward: one rank's rows of 8 sources, first product of an expert
        dict(product, name="product_prefill_32768", entries=32768, rows=16384, skew=0.4),
        # training, a small odd batch of narrow experts: gradient of the first product's rows
        dict(op="rows_grad", name="rows_grad_777", experts=8, entries=777, rows=777, cols=520, hidden=1000, out="fp32",
             gather=False, weighted=False, skew=0.4),
        # training, a large batch: gradient of the second product's rows, from the tokens' gradients (gathered)
        dict(op="rows_grad", name="rows_grad_16384", experts=32, entries=16384, rows=8192, cols=7168, hidden=2048, out="bf16",
             gather=True, weighted=False, skew=0.4),
        # training, one more micro-batch of few rows added to fp32 gradients, some experts without a row
        dict(op="weights_grad", name="weights_grad_333_added", experts=16, entries=333, rows=100, cols=1024, hidden=1000,
             out="fp32", gather=True, base=True, skew=1.1),
        # training, a large batch: gradient of the first product's weights
        dict(op="weights_grad", name="weights_grad_16384", experts=32, entries=16384, rows=8192, cols=4096, hidden=7168,
             out="bf16", gather=True, base=False, skew=0.4),
        # decode: the activation between the two products of 64 entries
        dict(op="gate", name="gate_decode_64", entries=64, cols=2048, dtype="bf16", out="bf16", weighted=True, grad=False),
        # training: the activation's gradient, with that of the routing weights, over a large batch
        dict(op="gate", name="gate_grad_32768", entries=32768, cols=2048, dtype="bf16", out="bf16", weighted=True, grad=True),
        # int8 decode: 8 tokens' rows quantised, first product of an expert
        dict(op="int8", name="int8_decode_64", experts=32, entries=64, rows=8, cols=4096, hidden=7168, dtype="bf16", out="bf16",
             gated=False, weighted=False, skew=0.0),
        # int8, uneven groups: activation and quantisation in one, second product, weighted, fp32 sums
        dict(op="int8", name="int8_gated_2047", experts=32, entries=2047, rows=2047, cols=7168, hidden=2048, dtype="bf16",
             out="fp32", gated=True, weighted=True, skew=1.1),
        # int8 prefill
        dict(op="int8", name="int8_prefill_32768", experts=32, entries=32768, rows=16384, cols=4096, hidden=7168, dtype="bf16",
             out="bf16", gated=False, weighted=False, skew=0.4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "rows_grad", "weights_grad", "gate", "int8"])
    if op == "gate":
        cols = 8 * _log(rng, 1, 1000)
        return dict(op=op, entries=max(1, min(_log(rng, 1, 40000), (100 << 20) // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "fp32"]), out=rng.choice(["bf16", "fp32"]), weighted=rng.random() < 0.7,
                    grad=rng.random() < 0.5)
    entries, each = _log(rng, 1, 16000), rng.choice([1, 2, 8])
    case = dict(op=op, experts=_log(rng, 1, 48), entries=entries, rows=max(1, entries // each), cols=8 * _log(rng, 1, 512),
                hidden=8 * _log(rng, 2, 512), out=rng.choice(["bf16", "fp32"]), skew=rng.choice([0.0, 0.4, 1.1]))
    if op == "int8":
        case.update(hidden=16 * _log(rng, 1, 256), dtype=rng.choice(["bf16", "fp32"]), gated=rng.random() < 0.4,
                    weighted=rng.random() < 0.5)
        return case
    case["gather"] = rng.random() < 0.6
    if op == "weights_grad":
        return dict(case, base=rng.random() < 0.4)
    return dict(case, weighted=rng.random() < 0.4)


# ---- inputs -------------------------------------------------------------------------------------------------------


def _popularity(n, skew):
    p = torch.arange(1, n + 1, dtype=torch.float32, device="cuda") ** -skew
    return p / p.sum()


def _groups(c, g, st):
    """Entries of (row, expert) pairs sorted by expert, experts popular and rare."""
    E, n, R = c["experts"], c["entries"], c["rows"]
    e = torch.multinomial(_popularity(E, c["skew"])[torch.randperm(E, device="cuda", generator=g)], n, True, generator=g)
    row = torch.randint(R, (n,), device="cuda", generator=g)
    order = torch.argsort(e * R + row, stable=True)
    counts = torch.bincount(e, minlength=E)
    st["most"] = int(counts.max())  # the plain form pads every group to this
    st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    st["entry_row"] = row[order].to(torch.int32) if c.get("gather", not c.get("gated")) else None


def _experts(c, g, cols, hidden):
    """The experts' weights, one expert at a time (the 32-bit values of all would not be small)."""
    w = torch.empty(c["experts"], cols, hidden, dtype=torch.bfloat16, device="cuda")
    for i in range(c["experts"]):
        w[i] = 0.02 * torch.randn(cols, hidden, device="cuda", generator=g)
    return w


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    st = {"case": c}
    op, dev = c["op"], "cuda"
    n = c["entries"]

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=g)

    def outlying(rows, cols):  # a few outlier channels, tokens of different size
        x = normal(rows, cols)
        x *= 1.0 + 20.0 * (torch.rand(cols, device=dev, generator=g) < 0.01)
        x *= torch.exp(0.5 * normal(rows, 1))
        return x

    if op == "gate":
        st["most"], st["offsets"] = n, torch.tensor([0, n], dtype=torch.int32, device=dev)
        st["h"] = (1.5 * normal(n, 2 * c["cols"])).to(FLOAT[c["dtype"]])
        st["w"] = torch.rand(n, device=dev, generator=g) if c["weighted"] else None
        if c["grad"]:
            st["dout"] = (0.1 * normal(n, c["cols"])).to(FLOAT[c["out"]])
            st["dh"], st["dw"] = torch.zeros_like(st["h"]), torch.zeros(n, device=dev)
        else:
            st["out"] = torch.zeros(n, c["cols"], dtype=FLOAT[c["out"]], device=dev)
        return st
    E, N, H = c["experts"], c["cols"], c["hidden"]
    if not c.get("gather", not c.get("gated")):
        c["rows"] = n
    R = c["rows"]
    _groups(c, g, st)
    if op == "product":
        st["x"], st["b"] = outlying(R, H).bfloat16(), _experts(c, g, N, H)
        st["out"] = torch.zeros(n, N, dtype=FLOAT[c["out"]], device=dev)
    elif op == "rows_grad":
        st["x"], st["b"] = (0.1 * normal(R, N)).bfloat16(), _experts(c, g, N, H)
        st["out"] = torch.zeros(n, H, dtype=FLOAT[c["out"]], device=dev)
    elif op == "weights_grad":  # the rows are gathered, the outputs' gradients lie by entry
        st["x"], st["dout"] = outlying(R, H).bfloat16(), (0.1 * normal(n, N)).bfloat16()
        st["base"] = normal(E, N, H).to(FLOAT[c["out"]]) if c["base"] else None
        st["out"] = torch.zeros(E, N, H, dtype=FLOAT[c["out"]], device=dev)
        return st
    else:
        if c["gated"]:
            st["x"] = (1.5 * normal(n, 2 * H)).to(FLOAT[c["dtype"]])
        else:
            st["x"] = outlying(R, H).to(FLOAT[c["dtype"]])
        st["b"] = torch.empty(E, N, H, dtype=torch.int8, device=dev)
        st["bs"] = torch.empty(E, N, device=dev)
        for i in range(E):
            st["b"][i], st["bs"][i] = _to_int8(0.02 * normal(N, H))
        st["q"] = torch.zeros(R, H, dtype=torch.int8, device=dev)
        st["qs"] = torch.zeros(R, device=dev)
        st["out"] = torch.zeros(n, N, dtype=FLOAT[c["out"]], device=dev)
    st["w"] = torch.rand(n, device=dev, generator=g) if c["weighted"] else None
    return st


# ---- the plain forms ----------------------------------------------------------------------------------------------


def _to_int8(x):
    """Rows as int8 and a scale per row: the largest magnitude is worth 127."""
    v = x.float()
    scale = v.abs().amax(1) / 127.0
    q = torch.round(v / scale[:, None]).clamp(-127, 127)
    return torch.where(scale[:, None] > 0, q, 0.0).to(torch.int8), scale


def _gate(h, w):
    g, u = h.chunk(2, dim=1)
    a = g * (1.0 / (1.0 + torch.exp(-g))) * u
    return a if w is None else a * w[:, None]


def _gate_grad(h, w, dout):
    g, u = h.float().chunk(2, dim=1)
    d = dout.float()
    s = 1.0 / (1.0 + torch.exp(-g))
    dw = (d * g * s * u).sum(1)
    if w is not None:
        d = d * w[:, None]
    return torch.cat([d * u * s * (1.0 + g * (1.0 - s)), d * g * s], dim=1).to(h.dtype), dw


def _padded(st, n):
    """Every group padded to the largest: entries [E][most], which of them there are."""
    at = st["offsets"][:-1, None] + torch.arange(st["most"], device="cuda")
    ok = at < st["offsets"][1:, None]
    return at.clamp_max(n - 1).long(), ok


def _scatter(v, at, ok, n, w, dtype):
    if w is not None:
        v = v * w[at][..., None]
    at = torch.where(ok, at, n).view(-1)  # the padding goes to a row of its own
    out = torch.empty(n + 1, v.shape[-1], dtype=dtype, device=v.device)
    return out.index_copy_(0, at, v.to(dtype).view(-1, v.shape[-1]))[:n]


def _rows_of(x, st, at, ok):
    row = at if st["entry_row"] is None else st["entry_row"][at].long()
    return torch.where(ok[..., None], x[row].float(), 0.0)


def _plain(st):
    c = st["case"]
    op, n = c["op"], c["entries"]
    if op == "gate":
        if c["grad"]:
            return dict(zip(("dh", "dw"), _gate_grad(st["h"], st["w"], st["dout"])))
        return {"out": _gate(st["h"].float(), st["w"]).to(FLOAT[c["out"]])}
    at, ok = _padded(st, n)
    if op in ("product", "rows_grad"):
        b = st["b"].float()
        if op == "product":
            b = b.transpose(1, 2).contiguous()
        return {"out": _scatter(torch.bmm(_rows_of(st["x"], st, at, ok), b), at, ok, n, st["w"], FLOAT[c["out"]])}
    if op == "weights_grad":
        d = torch.where(ok[..., None], st["dout"][at].float(), 0.0).transpose(1, 2).contiguous()
        v = torch.bmm(d, _rows_of(st["x"], st, at, ok))
        if st["base"] is not None:
            v += st["base"].float()
        return {"out": v.to(FLOAT[c["out"]])}
    # 64 bits: the last bit of an activation next to a border decides a code
    q, scale = _to_int8(_gate(st["x"].double(), None).float() if c["gated"] else st["x"])
    # 32-bit floats hold the sums of products below 2^24 as they are; beyond they round like any fp32 sum
    v = torch.bmm(_rows_of(q, st, at, ok), st["b"].float().transpose(1, 2).contiguous())
    row = at if st["entry_row"] is None else st["entry_row"][at].long()
    v = v * scale[row][..., None] * st["bs"][:, None, :]
    return {"out": _scatter(v, at, ok, n, st["w"], FLOAT[c["out"]])}


# ---- the library's calls ------------------------------------------------------------------------------------------


def _calls(st):
    """The calls of one pass, their arguments marshalled once for the state's fixed buffers, as a serving or training
    loop keeps them."""
    import combine_count_amd as epdc
    c = st["case"]
    op, n = c["op"], c["entries"]
    kind = {"bf16": epdc.EPDC_BF16, "fp32": epdc.EPDC_FP32}
    out = kind[c["out"]]
    if op == "gate":
        dtype = kind[c["dtype"]]
        if c["grad"]:
            return [epdc.prepare_expert_gate_grad(1, c["cols"], n, dtype, st["h"], st["offsets"], st["w"], st["dout"], out,
                                                  st["dh"], st["dw"])]
        return [epdc.prepare_expert_gate(1, c["cols"], n, dtype, st["h"], st["offsets"], st["w"], st["out"], out)]
    E, N, H, R = c["experts"], c["cols"], c["hidden"], c["rows"]
    if op == "product":
        return [epdc.prepare_expert_linear(E, N, H, n, R, st["x"], st["offsets"], st["entry_row"], st["w"], st["b"],
                                                 st["out"], out)]
    if op == "rows_grad":
        return [epdc.prepare_expert_rows_grad(E, N, H, n, R, st["x"], st["offsets"], st["entry_row"], st["w"], st["b"],
                                              st["out"], out)]
    if op == "weights_grad":
        return [epdc.prepare_expert_weights_grad(E, N, H, n, n, st["dout"], None, R, st["x"], st["entry_row"], st["offsets"],
                                                 st["base"], st["out"], out)]
    if c["gated"]:
        first = epdc.prepare_expert_gate_int(E, H, n, kind[c["dtype"]], st["x"], st["offsets"], None, st["q"], st["qs"])
    else:
        first = epdc.prepare_int_quantize(1, R, H, kind[c["dtype"]], st["x"], None, st["q"], st["qs"])
    return [first, epdc.prepare_expert_linear_int(E, N, H, n, R, st["q"], st["qs"], st["offsets"], st["entry_row"], st["w"],
                                                    st["b"], st["bs"], st["out"], out)]


def run(st):
    if not own:
        return _plain(st)
    if "calls" not in st:
        st["calls"] = _calls(st)
    for call in st["calls"]:
        call()
    return {"dh": st["dh"], "dw": st["dw"]} if "dh" in st else {"out": st["out"]}


# ---- what a pass cannot do without --------------------------------------------------------------------------------


def work(case):
    c = case
    op, n = c["op"], c["entries"]
    if op == "gate":
        F, d, o = c["cols"], SIZE[c["dtype"]], SIZE[c["out"]]
        if c["grad"]:
            return {"bytes": n * F * (4 * d + o) + n * (8 if c["weighted"] else 4), "flops": 12 * n * F}
        return {"bytes": n * F * (2 * d + o) + (n * 4 if c["weighted"] else 0), "flops": 5 * n * F}
    E, N, H = c["experts"], c["cols"], c["hidden"]
    touched = E * (1.0 - (1.0 - 1.0 / E) ** n)  # experts with an entry
    R = min(n, c["rows"]) if c.get("gather", not c.get("gated")) else n
    if op == "weights_grad":
        return {"bytes": R * H * 2 + n * N * 2 + E * N * H * SIZE[c["out"]] * (2 if c["base"] else 1), "flops": 2 * n * N * H}
    if op == "int8":
        rows = n * 2 * H * SIZE[c["dtype"]] if c["gated"] else R * H * SIZE[c["dtype"]]
        return {"bytes": touched * N * (H + 4) + rows + n * N * SIZE[c["out"]], "flops": 2 * n * N * H}
    inner, outer = (H, N) if op == "product" else (N, H)
    return {"bytes": touched * N * H * 2 + R * inner * 2 + n * outer * SIZE[c["out"]], "flops": 2 * n * N * H}


# ---- 64 bits, from the definitions --------------------------------------------------------------------------------


def _exact_gate(h, w):
    h = h.double()
    F = h.shape[1] // 2
    a = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]
    return a if w is None else w.double()[:, None] * a


def _exact_int8(x):
    """x in 64 bits; the scale is a 32-bit number and so is the quotient that is rounded to a whole one."""
    scale = (x.abs().max(dim=1).values.float().double() / 127.0).float().double()
    q = (x.float().double() / scale[:, None]).float().double()
    low = torch.floor(q)
    up = (q - low > 0.5) | ((q - low == 0.5) & (low % 2 != 0))  # a half goes to the even one
    return torch.where(scale[:, None] > 0, low + up, 0.0).clamp(-127, 127), scale


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    op, n = c["op"], c["entries"]
    if op == "gate" and c["grad"]:  # by automatic differentiation
        h = st["h"].double().requires_grad_(True)
        w = (torch.ones(n, device="cuda") if st["w"] is None else st["w"]).double().requires_grad_(True)
        (_exact_gate(h, w) * st["dout"].double()).sum().backward()
        return {"dh": h.grad, "dw": w.grad}
    if op == "gate":
        return {"out": _exact_gate(st["h"], st["w"])}
    bounds = st["offsets"].tolist()
    if op == "int8":
        a, scale = _exact_int8(_exact_gate(st["x"], None) if c["gated"] else st["x"].double())
        a = a * scale[:, None]
    else:
        a = st["x"].double()
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        rows = a[lo:hi] if st["entry_row"] is None else a[st["entry_row"][lo:hi].long()]
        if op == "weights_grad":
            out[e] = st["dout"][lo:hi].double().t().contiguous() @ rows
            if st["base"] is not None:
                out[e] += st["base"][e]
        elif lo < hi:
            b = st["b"][e].double()
            if op == "int8":
                b = b * st["bs"][e].double()[:, None]
            out[lo:hi] = rows @ (b if op == "rows_grad" else b.t().contiguous())
    if st.get("w") is not None:
        out *= st["w"].double()[:, None]
    return {"out": out}
