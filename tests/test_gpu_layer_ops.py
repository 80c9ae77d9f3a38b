"""Routing and its gradient, fp4x2 quantisation, grouping by expert and the
experts' product on the GPU, against the 64-bit implementations of
layer_oracle.py.  What is chosen, counted, copied or quantised has to be
equal; the tolerance of a computed number is derived where it is used, in
half steps of its type (a rounding is off by at most half a step)."""
import numpy as np
import pytest
import torch

import combine_count_amd as epdc
import layer_oracle as oracle

pytestmark = pytest.mark.gpu

INF = float("inf")
HALF32 = 2.0 ** -24
KIND = {"bf16": (epdc.EPDC_BF16, torch.bfloat16), "fp32": (epdc.EPDC_FP32, torch.float32)}
HALF = {"bf16": 2.0 ** -8, "fp32": HALF32}  # half a step, relative
TINY = {"bf16": 2.0 ** -134, "fp32": 2.0 ** -150}  # half a step of the smallest subnormal


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda") if dtype is None else torch.as_tensor(a).to("cuda", dtype)


# ---- routing ------------------------------------------------------------------------------------------------------

ROUTES = [
    # (experts, topk, groups, kept, groupTop, score, bias, renorm)
    (256, 8, 8, 4, 2, "sigmoid", True, True),
    (256, 8, 1, 1, 1, "softmax", False, True),
    (256, 8, 1, 1, 1, "softmax", True, False),
    (128, 6, 1, 1, 1, "softmax", False, False),
    (64, 8, 8, 3, 1, "softmax", False, True),
    (160, 6, 8, 3, 1, "softmax", True, True),
    (60, 4, 1, 1, 1, "sigmoid", True, False),
    (60, 4, 4, 2, 2, "sigmoid", False, True),
    (77, 5, 7, 3, 2, "sigmoid", True, True),
    (384, 8, 1, 1, 1, "sigmoid", True, True),
    (512, 10, 16, 4, 2, "softmax", True, True),
    (1024, 64, 64, 32, 2, "sigmoid", True, True),
    (1000, 17, 1, 1, 1, "softmax", False, False),
    (8, 8, 4, 4, 1, "softmax", False, True),
    (16, 1, 1, 1, 1, "softmax", False, False),
    (48, 16, 3, 1, 2, "sigmoid", True, False),
    (256, 16, 8, 8, 1, "sigmoid", True, True),
    (1, 1, 1, 1, 1, "softmax", False, True),
    (3, 2, 3, 2, 1, "sigmoid", True, True),
    (200, 9, 2, 1, 2, "softmax", True, True),
]
VALUES = ["normal", "ties", "masked", "wide"]


def logits_of(values, T, E, dtype, rng):
    l = rng.standard_normal((T, E))
    if values == "ties":  # a handful of values: nearly every comparison is a tie
        l = rng.integers(-2, 3, (T, E)).astype(np.float64)
        l[:, ::5] = -0.0
    elif values == "masked":
        l[rng.random((T, E)) < 0.5] = -INF
        l[rng.random((T, E)) < 0.05] = np.nan
        l[rng.random(T) < 0.3] = -INF  # nothing left to choose
        l[0] = np.nan
        if T > 2:
            l[1] = -INF
            l[1, E // 2] = 0.5  # one expert left
    elif values == "wide":
        l *= 40.0
        l[rng.random((T, E)) < 0.1] = float(torch.finfo(KIND[dtype][1]).min)
        l[rng.random((T, E)) < 0.01] = INF
        l[rng.random((T, E)) < 0.1] = -INF
    t = torch.from_numpy(l).to(KIND[dtype][1])
    return t, t.double().numpy()


def run_route(E, K, G, keep, top, score, renorm, scale, dtype, l, bias, stream=None):
    T = l.shape[0]
    cfg = epdc.RouteCfg(E, K, KIND[dtype][0], epdc.EPDC_SOFTMAX if score == "softmax" else epdc.EPDC_SIGMOID, G, keep, top,
                        int(renorm), scale)
    ids = torch.full((T + 1, K), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, K), -7.0, device="cuda")
    epdc.epdc_route(cfg, T, l, bias, ids, w, stream=stream)
    torch.cuda.synchronize()
    assert bool((ids[T] == -77).all()) and bool((w[T] == -7.0).all())  # nothing behind the last token
    return ids[:T].cpu().numpy(), w[:T].double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("values", VALUES)
@pytest.mark.parametrize("cfg", ROUTES, ids=lambda c: "-".join(map(str, c)))
def test_route(cfg, values, dtype):
    E, K, G, keep, top, score, biased, renorm = cfg
    rng = np.random.default_rng(E * 1000 + K)
    T, scale = 37, 2.5
    t, l = logits_of(values, T, E, dtype, rng)
    bias = None
    if biased:
        bias = (0.2 * rng.standard_normal(E)).astype(np.float32)
        if values == "masked" and E > 4:
            bias[1], bias[2], bias[3] = -INF, np.nan, INF
        if values == "ties":
            bias[:] = np.float32(0.25) * rng.integers(0, 2, E)
    ids, w = run_route(E, K, G, keep, top, score, renorm, scale, dtype, t.cuda(), None if bias is None else dev(bias))
    want_ids, want = oracle.route(l, bias, K, score == "softmax", G, keep, top, renorm, scale)
    np.testing.assert_array_equal(ids, want_ids)
    # computed in 64 bits and rounded once: half a step, and what 64 bits are off themselves
    assert np.all(np.abs(w - want) <= HALF32 * (1 + 2.0 ** -20) * np.abs(want) + TINY["fp32"])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,G,keep,top", [(200, 256, 8, 8, 4, 2), (2100, 256, 8, 8, 4, 2), (200, 256, 8, 1, 1, 1),
                                              (2100, 256, 8, 1, 1, 1), (200, 96, 6, 4, 2, 2), (200, 128, 6, 4, 2, 2),
                                              (200, 500, 20, 1, 1, 1)])
def test_route_decides_near_ties_in_64_bits(T, E, K, G, keep, top, score):
    """Choice values a few 2^-26 apart: equal or reversed in 32 bits."""
    rng = np.random.default_rng(5)
    base = rng.standard_normal((T, 1)) * 0.5 + 1.0
    l = (base + rng.integers(-3, 4, (T, E)) * 2.0 ** -23).astype(np.float32)
    bias = (rng.integers(-3, 4, E) * 2.0 ** -26).astype(np.float32)
    ids, w = run_route(E, K, G, keep, top, score, True, 1.0, "fp32", dev(l), dev(bias))
    want_ids, want = oracle.route(l, bias, K, score == "softmax", G, keep, top, True, 1.0)
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= HALF32 * (1 + 2.0 ** -20) * np.abs(want))


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,K", [(2048, 64), (300, 63), (2100, 64), (2100, 15), (2100, 16)])
def test_route_of_as_many_experts_as_there_are_lanes(T, K, biased):
    """The last choice and the first left out, closer than 32-bit words with the expert's number in them tell."""
    rng = np.random.default_rng(K)
    l = (rng.integers(-8, 8, (T, 256)) * 0.25 + rng.integers(0, 64, (T, 256)) * 2.0 ** -20).astype(np.float32)
    bias = (0.25 * rng.integers(0, 2, 256)).astype(np.float32) if biased else None
    ids, w = run_route(256, K, 1, 1, 1, "sigmoid", True, 1.0, "fp32", dev(l), None if bias is None else dev(bias))
    want_ids, want = oracle.route(l, bias, K, False, 1, 1, 1, True, 1.0)
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= HALF32 * (1 + 2.0 ** -20) * np.abs(want))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [9, 2100])
def test_route_groups_of_the_lowest_bias(T, dtype):
    """Experts put out of reach by the lowest fp32 number are not masked: a group of them goes before a masked group,
    and behind a group with one ordinary expert."""
    rng = np.random.default_rng(T)
    t, l = logits_of("normal", T, 256, dtype, rng)
    bias = np.full(256, np.finfo(np.float32).min, dtype=np.float32)
    bias[0:32] = -INF      # group 0: nothing
    bias[40] = 0.5         # group 1: one ordinary expert
    bias[96:128] = 0.25    # group 3: ordinary
    bias[128] = -3e38      # group 4: a little better than 2, 5, 6 and 7
    for keep in (3, 4, 7):
        ids, _ = run_route(256, 12, 8, keep, 2, "sigmoid", True, 1.0, dtype, t.cuda(), dev(bias))
        np.testing.assert_array_equal(ids, oracle.route(l, bias, 12, False, 8, keep, 2, True, 1.0)[0])


@pytest.mark.parametrize("T,values", [(0, "normal"), (1, "normal"), (2, "normal"), (3, "normal"), (5, "normal"), (64, "normal"),
                                      (65, "normal"), (1023, "normal"), (2048, "normal"), (2049, "normal"), (2051, "masked"),
                                      (2050, "ties"), (2055, "wide")])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_token_counts(T, values, dtype):
    rng = np.random.default_rng(T)
    t, l = logits_of(values, T, 256, dtype, rng)
    bias = (0.1 * rng.standard_normal(256)).astype(np.float32)
    ids, w = run_route(256, 8, 8, 4, 2, "sigmoid", True, 1.0, dtype, t.cuda(), dev(bias))
    want_ids, want = oracle.route(l, bias, 8, False, 8, 4, 2, True, 1.0)
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= HALF32 * (1 + 2.0 ** -20) * want + TINY["fp32"])


@pytest.mark.parametrize("dtype,skip", [("bf16", 1), ("bf16", 4), ("fp32", 1), ("fp32", 2)])
def test_route_from_an_odd_address(dtype, skip):
    """Logits that start between 16-byte borders."""
    rng = np.random.default_rng(3)
    T, E = 19, 256
    t, l = logits_of("normal", T, E, dtype, rng)
    buf = torch.zeros(T * E + 8, dtype=t.dtype, device="cuda")
    buf[skip:skip + T * E] = t.reshape(-1).cuda()
    view = buf[skip:skip + T * E].view(T, E)
    ids, _ = run_route(E, 8, 8, 4, 2, "sigmoid", True, 1.0, dtype, view, None)
    np.testing.assert_array_equal(ids, oracle.route(l, None, 8, False, 8, 4, 2, True, 1.0)[0])
    dw = rng.standard_normal((T, 8)).astype(np.float32)
    out = torch.zeros(T * E + 8, dtype=t.dtype, device="cuda")
    got = run_grad(E, 8, "softmax", False, 1.0, dtype, view, ids, dw, out[skip:skip + T * E].view(T, E))
    check_grad(got, l, ids, dw, "softmax", False, 1.0, dtype)
    assert bool((out[:skip] == 0).all()) and bool((out[skip + T * E:] == 0).all())


# ---- the gradient -------------------------------------------------------------------------------------------------


def run_grad(E, K, score, renorm, scale, dtype, l, ids, dw, out=None):
    T = l.shape[0]
    cfg = epdc.RouteCfg(E, K, KIND[dtype][0], epdc.EPDC_SOFTMAX if score == "softmax" else epdc.EPDC_SIGMOID, 1, 1, 1,
                        int(renorm), scale)
    if out is None:
        out = torch.full((T, E), 9.0, dtype=KIND[dtype][1], device="cuda")
    epdc.epdc_route_grad(cfg, T, l, dev(ids), dev(dw), out)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


def check_grad(got, l, ids, dw, score, renorm, scale, dtype):
    want, mag = oracle.route_grad(l, ids, dw, score == "softmax", renorm, scale)
    # Half steps of 32 bits, relative to the magnitudes summed: an exponential (at most 2 ulp, 4 half steps) of an
    # argument off by half a step of itself (up to its size), in numerator, sum and (1 - s) each; sums of up to 64
    # terms over lanes (6) and 16 in a lane; division (up to 5 half steps) and 8 products.  Then one rounding of the
    # result, and half a step of the smallest subnormal for results that small (32-bit factors below 2^-126 lose up
    # to 2^-126 of themselves where the hardware's exponential flushes).
    finite = np.where(np.isfinite(l), l, 0.0)
    size = np.minimum(np.abs(finite).max(1, keepdims=True) * 2, 110.0)
    steps = 3 * (4 + size) + 6 + 16 + 3 * 5 + 8 + ids.shape[1]
    bound = steps * HALF32 * mag + (HALF[dtype] if dtype == "bf16" else 0.0) * np.abs(want) + TINY[dtype]
    bound += 2.0 ** -125 * (np.abs(dw).max() if dw.size else 0.0) * abs(scale) * 2
    bad = np.abs(got - want) > bound
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], bound[bad][:5])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("E,K,T,values", [
    (256, 8, 33, "normal"), (128, 6, 5, "normal"), (256, 8, 29, "masked"), (256, 8, 29, "wide"), (60, 4, 7, "ties"),
    (77, 5, 9, "masked"), (1000, 64, 6, "normal"), (1024, 9, 6, "wide"), (1, 1, 3, "normal"), (8, 8, 1, "normal"),
    (384, 8, 4, "wide"), (512, 16, 130, "normal"), (264, 3, 5, "masked")])
def test_route_grad(E, K, T, values, score, renorm, dtype):
    rng = np.random.default_rng(E + K)
    t, l = logits_of(values, T, E, dtype, rng)
    ids = oracle.route(l, None, K, score == "softmax")[0]
    ids[rng.random(ids.shape) < 0.1] = -1  # dropped slots
    if T > 3:
        ids[2] = -1
        ids[3, 0] = E + 5  # no expert
    dw = rng.standard_normal((T, K)).astype(np.float32)
    got = run_grad(E, K, score, renorm, 2.5, dtype, t.cuda(), ids, dw)
    check_grad(got, l, ids, dw, score, renorm, 2.5, dtype)


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_route_grad_adds_up_the_slots_of_one_expert(score, renorm):
    rng = np.random.default_rng(11)
    T, E, K = 21, 96, 6
    t, l = logits_of("normal", T, E, "fp32", rng)
    ids = rng.integers(0, 4, (T, K)).astype(np.int32)  # every token has slots of the same expert
    dw = rng.standard_normal((T, K)).astype(np.float32)
    got = run_grad(E, K, score, renorm, 1.5, "fp32", t.cuda(), ids, dw)
    check_grad(got, l, ids, dw, score, renorm, 1.5, "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [64, 96, 128, 256])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_route_grad_of_slots_that_hold_masked_experts(score, renorm, E, dtype):
    rng = np.random.default_rng(E)
    T, K = 23, 5
    t, _ = logits_of("normal", T, E, dtype, rng)
    t[:, 3], t[:, 4] = np.nan, -INF
    ids = rng.integers(5, E, (T, K)).astype(np.int32)
    ids[::2, 1], ids[1::3, 2], ids[5] = 3, 4, 3
    dw = rng.standard_normal((T, K)).astype(np.float32)
    dw[0, 1] = np.nan  # and whatever its gradient is
    got = run_grad(E, K, score, renorm, 1.5, dtype, t.cuda(), ids, dw)
    check_grad(got, t.double().numpy(), ids, np.where(np.isnan(dw), 0, dw), score, renorm, 1.5, dtype)


@pytest.mark.parametrize("E", [96, 128])
def test_route_grad_of_scores_below_32_bits(E):
    """Renormalised sigmoids of which no 32-bit value is left: their shares are (0 where 64 bits leave none either)."""
    rng = np.random.default_rng(E)
    T, K = 40, 6
    l = (rng.standard_normal((T, E)) - 90.0 - 20.0 * np.arange(T)[:, None]).astype(np.float32)
    ids = oracle.route(l, None, K, False)[0]
    dw = rng.standard_normal((T, K)).astype(np.float32)
    got = run_grad(E, K, "sigmoid", True, 1.5, "fp32", dev(l), ids, dw)
    assert np.abs(got[:30]).max(1).min() > 1e-3 and not got[32:].any()
    check_grad(got, l.astype(np.float64), ids, dw, "sigmoid", True, 1.5, "fp32")


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_route_grad_against_differences(score, renorm):
    """d(sum of weights * dw) along a direction, by central differences of the 64-bit weights."""
    rng = np.random.default_rng(7)
    T, E, K, scale, h = 16, 64, 4, 2.5, 1e-4
    t, l = logits_of("normal", T, E, "fp32", rng)
    ids = oracle.route(l, None, K, score == "softmax")[0]
    dw = rng.standard_normal((T, K)).astype(np.float32)
    got = run_grad(E, K, score, renorm, scale, "fp32", t.cuda(), ids, dw)
    for _ in range(4):
        d = rng.standard_normal((T, E))
        f = [(oracle.weights_of(l + s * h * d, ids, score == "softmax", renorm, scale) * dw).sum(1) for s in (1, -1)]
        slope = (f[0] - f[1]) / (2 * h)
        # the third derivative along d: scores' third derivatives are below 1 in size, |d_i| <= 5, so
        # h^2/6 * scale * sum |dw| * (sum of |d| over the experts that matter)^3, well under 1e-4 here; 32 bits add
        # under 1e-5
        assert np.all(np.abs((got * d).sum(1) - slope) <= 1e-4 * scale * (1 + np.abs(dw).sum(1)))


# ---- fp4x2 rows ---------------------------------------------------------------------------------------------------


def quantize(x, cols, dtype, W=1, count=None):
    """x [W][M][cols]; the outputs pre-filled, so that what is not written shows."""
    M = x.shape[0] * x.shape[1] // W if x.dim() == 3 else x.shape[0] // W
    q = torch.full((W * M, cols // 2), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((W * M, epdc.epdc_mx_scale_dim(cols)), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    epdc.epdc_mx_quantize(W, M, cols, KIND[dtype][0], x, None if count is None else dev(count, torch.int32), q, s)
    torch.cuda.synchronize()
    return q, s


def check_quantized(q, s, x64):
    want_q, want_s = oracle.pack(*oracle.mx_quantize(x64))
    np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (7, 96), (5, 160), (1, 7168), (130, 2048), (33, 1056), (2, 131072)])
def test_mx_quantize(rows, cols, dtype):
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1)))
    x[:, ::7] *= 30.0
    if rows > 2:
        x[1] = 0.0
    t = torch.from_numpy(x).to(KIND[dtype][1])
    q, s = quantize(t.cuda(), cols, dtype)
    check_quantized(q, s, t.double().numpy())


def test_mx_quantize_every_bf16():
    """Every bf16 value as the largest of its block, next to smaller ones over 32 powers of two of every kind."""
    bits = np.arange(65536, dtype=np.uint32)
    first = (bits << 16).view(np.float32).astype(np.float64)
    rng = np.random.default_rng(1)
    with np.errstate(all="ignore"):
        block = first[:, None] * np.concatenate([[1.0], rng.uniform(-1, 1, 15), np.exp2(-np.arange(16.0))])
    t = torch.from_numpy(block).to(torch.bfloat16)
    q, s = quantize(t.cuda(), 32, "bf16")
    check_quantized(q, s, t.double().numpy())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_mx_quantize_ties_subnormals_and_the_largest(dtype):
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.5, 0.0, 6.0, 7.9375])
    ties = np.concatenate([ties, -ties, [4.0] * 8])
    x = np.stack([ties * 2.0 ** e for e in list(range(-126, 126)) + [-140, -133, -130, -127]])
    x[:, -1] = 4.0 * np.exp2(np.array(list(range(-126, 126)) + [-140, -133, -130, -127], dtype=np.float64))
    t = torch.from_numpy(x).to(KIND[dtype][1])
    q, s = quantize(t.cuda(), 32, dtype)
    check_quantized(q, s, t.double().numpy())
    if dtype == "fp32":  # beside a tie: one step of 32 bits to either side
        near = np.nextafter(x.astype(np.float32), np.float32(np.inf)).astype(np.float64)
        near = np.concatenate([near, np.nextafter(x.astype(np.float32), np.float32(-np.inf)).astype(np.float64)])
        t = torch.from_numpy(near).float()
        q, s = quantize(t.cuda(), 32, dtype)
        check_quantized(q, s, t.double().numpy())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_mx_blocks_that_are_not_finite(dtype):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((6, 128))
    x[0, 3], x[1, 40], x[2, 127], x[3, 0] = np.nan, INF, -INF, float(torch.finfo(KIND[dtype][1]).max)
    t = torch.from_numpy(x).to(KIND[dtype][1])
    q, s = quantize(t.cuda(), 128, dtype)
    check_quantized(q, s, t.double().numpy())
    out = torch.empty(6, 128, dtype=torch.float32, device="cuda")
    epdc.epdc_mx_dequantize(1, 6, 128, q, s, None, out, epdc.EPDC_FP32)
    torch.cuda.synchronize()
    got = out.cpu().numpy()
    assert np.isnan(got[0, :32]).all() and np.isnan(got[1, 32:64]).all() and np.isnan(got[2, 96:]).all()
    assert np.isfinite(got).sum() == 6 * 128 - 96


@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_mx_dequantize_every_code_and_scale(out):
    codes = np.tile(np.arange(16, dtype=np.uint8), 256 * 2).reshape(256, 32)
    byte = np.arange(256, dtype=np.uint8)[:, None]
    q, s = oracle.pack(codes, byte)
    o = torch.full((257, 32), 7.0, dtype=KIND[out][1], device="cuda")
    epdc.epdc_mx_dequantize(1, 256, 32, dev(q), dev(s), None, o, KIND[out][0])
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(oracle.mx_values(codes, byte)).to(KIND[out][1])
    got = o[:256].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[:255], want[:255])
    assert torch.equal(torch.signbit(got[:255]), torch.signbit(want[:255]))
    assert bool((o[256] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("W,M,cols,count", [(4, 37, 160, [0, 37, 5, 36]), (3, 300, 2048, [300, 1, 299]), (2, 5, 32, [-3, 99]),
                                            (1, 64, 7168, [17])])
def test_mx_windows_leave_the_other_rows(W, M, cols, count, dtype):
    rng = np.random.default_rng(cols)
    t = torch.from_numpy(rng.standard_normal((W, M, cols))).to(KIND[dtype][1])
    q, s = quantize(t.cuda(), cols, dtype, W, np.array(count))
    live = (np.arange(M)[None] < np.array(count)[:, None]).reshape(-1)
    want_q, want_s = oracle.pack(*oracle.mx_quantize(t.double().numpy().reshape(-1, cols)))
    want_q[~live], want_s[~live] = 0xA5, 0x5A5A5A5A
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    o = torch.full((W * M, cols), 7.0, dtype=KIND[dtype][1], device="cuda")
    epdc.epdc_mx_dequantize(W, M, cols, q, s, dev(np.array(count), torch.int32), o, KIND[dtype][0])
    torch.cuda.synchronize()
    got = o.double().cpu().numpy()
    want = oracle.mx_values(*oracle.unpack(want_q[live], want_s[live]))
    np.testing.assert_array_equal(got[live], want)
    assert (got[~live] == 7.0).all()


# ---- grouping -----------------------------------------------------------------------------------------------------


def run_group(W, M, epr, K, rank, ids, count, weights=True, stream=None):
    cfg = epdc.EpCfg(W, 1024, M, epr, K, epdc.EPDC_BF16, int(weights), 0)
    groups = (W if rank < 0 else 1) * epr
    rng = np.random.default_rng(0)
    w = rng.random(ids.shape).astype(np.float32)
    out = dict(offsets=torch.full((groups + 1,), -5, dtype=torch.int32, device="cuda"),
               row=torch.full((ids.size,), -6, dtype=torch.int32, device="cuda"),
               weight=torch.full((ids.size,), -7.0, device="cuda"),
               of=torch.full(ids.shape, -8, dtype=torch.int32, device="cuda"))
    scratch = torch.full((epdc.epdc_group_scratch_bytes(cfg, rank) // 4,), 12345, dtype=torch.int32, device="cuda")
    epdc.epdc_group_experts(cfg, rank, dev(ids), dev(w) if weights else None, None if count is None else dev(count, torch.int32),
                            out["offsets"], out["row"], out["weight"] if weights else None, out["of"], scratch, stream=stream)
    torch.cuda.synchronize()
    return w, {k: v.cpu().numpy() for k, v in out.items()}


def check_group(W, M, epr, K, rank, ids, count, weights=True):
    w, got = run_group(W, M, epr, K, rank, ids, count, weights)
    offsets, row, slots, of = oracle.group(ids, np.full(W, M) if count is None else count, epr, rank)
    np.testing.assert_array_equal(got["offsets"], offsets)
    n = offsets[-1]
    np.testing.assert_array_equal(got["row"][:n], row)
    assert (got["row"][n:] == -6).all()  # left as they were
    np.testing.assert_array_equal(got["of"], of)
    if weights:
        np.testing.assert_array_equal(got["weight"][:n], w.reshape(-1)[slots])
    assert (got["weight"][n if weights else 0:] == -7.0).all()


@pytest.mark.parametrize("W,M,epr,K,rank,fill", [
    (4, 8, 4, 2, -1, 0.7), (4, 8, 4, 2, 2, 0.7), (8, 128, 8, 8, -1, 0.6), (8, 128, 8, 8, 7, 1.0), (1, 1, 1, 1, 0, 1.0),
    (1, 1000, 64, 8, 0, 1.0), (3, 257, 33, 5, 1, 0.9), (8, 700, 32, 8, 3, 0.5), (8, 700, 32, 8, -1, 0.5), (2, 300, 1000, 7, 1, 0.9),
    (2, 33, 1024, 64, -1, 0.9), (64, 5, 2, 3, -1, 0.8), (1, 5000, 1, 1, 0, 0.99), (2, 2049, 3, 1, -1, 1.0), (5, 31, 7, 6, 4, 0.0),
    (16, 900, 40, 8, 5, 0.8), (16, 900, 40, 8, -1, 0.8),
    # above the words a block sums itself: the scan launches between
    (64, 260, 600, 8, 2, 0.9), (64, 260, 600, 8, -1, 0.9), (3, 4000, 1024, 8, 0, 0.9), (40, 300, 700, 1, -1, 0.9)])
def test_group(W, M, epr, K, rank, fill):
    rng = np.random.default_rng(W * 1000 + M)
    E = W * epr
    ids = rng.integers(0, E, (W, M, K)).astype(np.int32)
    if rank >= 0:  # most of them this rank's
        mine = rng.random(ids.shape) < 0.6
        ids = np.where(mine, rank * epr + ids % epr, ids).astype(np.int32)
    ids[rng.random(ids.shape) < 0.05] = -1
    ids[rng.random(ids.shape) < 0.02] = 2 ** 31 - 1
    ids[rng.random(ids.shape) < 0.02] = -2 ** 31
    count = np.minimum(np.round(rng.uniform(0.5, 1.5, W) * fill * M), M).astype(np.int32)
    check_group(W, M, epr, K, rank, ids, count)


def test_group_counts_out_of_range_all_rows_and_no_weights():
    rng = np.random.default_rng(4)
    ids = rng.integers(0, 12, (3, 70, 4)).astype(np.int32)
    check_group(3, 70, 4, 4, -1, ids, np.array([-5, 1000, 70], dtype=np.int32))
    check_group(3, 70, 4, 4, 1, ids, None)
    check_group(3, 70, 4, 4, 1, ids, np.array([70, 0, 69], dtype=np.int32), weights=False)
    check_group(3, 70, 4, 4, 2, np.full((3, 70, 4), 9, dtype=np.int32), None)  # one expert has them all
    check_group(3, 70, 4, 4, 2, np.full((3, 70, 4), 0, dtype=np.int32), None)  # none


# ---- the experts' product -----------------------------------------------------------------------------------------


def random_mx(rng, rows, cols):
    """Codes and scales of every kind, the scales within 2^-6 .. 2^6."""
    codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    byte = rng.integers(121, 134, (rows, cols // 32)).astype(np.uint8)
    return oracle.pack(codes, byte) + (oracle.mx_values(codes, byte),)


def sizes_to_offsets(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


def check_product(sizes, N, H, out, R=None, weighted=False, extra=0, rows=None, offsets=None, seed=0):
    """R: rows to gather from (None: entry i is row i)."""
    rng = np.random.default_rng(seed)
    E = len(sizes)
    offsets = sizes_to_offsets(sizes) if offsets is None else np.asarray(offsets, dtype=np.int32)
    n = int(offsets.max()) + extra
    a_rows = n if R is None else R
    aq, as_, a = random_mx(rng, a_rows, H)
    bq, bs, b = random_mx(rng, E * N, H)
    if R is not None and rows is None:
        rows = rng.integers(0, R, n).astype(np.int32)
    w = rng.standard_normal(n).astype(np.float32) if weighted else None
    o = torch.full((n, N), 77.0, dtype=KIND[out][1], device="cuda")
    epdc.epdc_expert_product(E, N, H, n, a_rows, dev(aq), dev(as_), dev(offsets), None if rows is None else dev(rows),
                             None if w is None else dev(w), dev(bq), dev(bs), o, KIND[out][0])
    torch.cuda.synchronize()
    got = o.double().cpu().numpy()
    want, mag = oracle.product(a, b.reshape(E, N, H), offsets, rows, w, n)
    none = np.isnan(want)
    assert (got[none] == 77.0).all()  # rows of no group are left as they were
    # H products exact in 32 bits, H additions in any order, the weight; a truncating addition is off by a whole
    # step: two half steps each; then the result's rounding
    bound = (2 * H + 4) * HALF32 * mag + HALF[out] * np.abs(want)
    bad = ~none & (np.abs(got - want) > np.where(none, 0, bound))
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes,N,H,R,weighted", [
    ([1], 16, 32, None, False), ([1, 0, 2], 8, 64, 5, True), ([5, 17, 0, 33], 64, 128, 40, False),
    ([16, 16], 128, 256, None, True), ([3, 100, 64, 1], 72, 96, 77, True), ([0, 0, 0], 64, 128, None, False),
    ([31, 32, 33], 200, 736, 50, False), ([2] * 40, 264, 1056, 16, True), ([129, 255, 257], 256, 512, 300, True),
    ([700], 136, 288, None, False), ([300, 0, 20, 513], 520, 1024, 900, False), ([64] * 8, 1024, 2048, 64, False),
    ([1] * 8, 2048, 7168, 8, True), ([8], 512, 7168, 8, False), ([1000, 1], 264, 160, 600, True),
    ([257, 128, 1, 640], 768, 1184, 700, True), ([512, 511], 1032, 384, None, True)])
def test_expert_product(sizes, N, H, R, weighted, out):
    if out == "bf16" and N * 2 % 16:
        pytest.skip("bf16 rows of 16 bytes")
    check_product(sizes, N, H, out, R, weighted, extra=3)


@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("steps", range(1, 12))
@pytest.mark.parametrize("tail", [0, 32, 128, 224])
def test_expert_product_every_number_of_steps(steps, tail, rows):
    """Rows of 1 to 11 steps of 256 elements, whole or ending inside the last."""
    check_product([rows, rows + 7], 136, 256 * steps - tail, "fp32", R=97, weighted=True, seed=steps)


def test_expert_product_rows_outside_and_odd_offsets():
    rows = np.array([0, -1, 5, 1000000, 3, -2 ** 31, 2 ** 31 - 1, 9] * 10, dtype=np.int32)
    check_product([30, 50], 64, 256, "fp32", R=10, rows=rows, weighted=True)
    # entries before the first group; groups that run backwards are empty; ends beyond maxEntries are cut
    check_product([0] * 3, 64, 256, "fp32", R=10, offsets=[5, 20, 12, 40], rows=rows[:40])
    rng = np.random.default_rng(0)
    aq, as_, a = random_mx(rng, 8, 64)
    bq, bs, b = random_mx(rng, 2 * 16, 64)
    o = torch.full((12, 16), 77.0, device="cuda")
    epdc.epdc_expert_product(2, 16, 64, 8, 8, dev(aq), dev(as_), dev(np.array([-4, 3, 2 ** 31 - 1], dtype=np.int32)), None, None,
                             dev(bq), dev(bs), o, epdc.EPDC_FP32)
    torch.cuda.synchronize()
    want, mag = oracle.product(a, b.reshape(2, 16, 64), np.array([0, 3, 8]), None, None, 8)
    assert np.all(np.abs(o[:8].double().cpu().numpy() - want) <= 132 * HALF32 * mag)
    assert bool((o[8:] == 77.0).all())


def test_expert_product_of_large_small_and_nan_scales():
    """Scales at both ends (their product still a 32-bit number), a NaN block reaches its row and column alone."""
    rng = np.random.default_rng(9)
    n, N, H = 40, 32, 256
    codes = rng.integers(0, 16, (n, H)).astype(np.uint8)
    byte = np.full((n, H // 32), 127, dtype=np.uint8)
    byte[:10], byte[10:20] = 240, 20
    bcodes = rng.integers(0, 16, (N, H)).astype(np.uint8)
    bbyte = np.full((N, H // 32), 127, dtype=np.uint8)
    bbyte[:8], bbyte[8:16] = 20, 110
    a, b = oracle.mx_values(codes, byte), oracle.mx_values(bcodes, bbyte)
    byte[30, 3], bbyte[20, 5] = 255, 255
    (aq, as_), (bq, bs) = oracle.pack(codes, byte), oracle.pack(bcodes, bbyte)
    o = torch.empty(n, N, device="cuda")
    epdc.epdc_expert_product(1, N, H, n, n, dev(aq), dev(as_), dev(np.array([0, n], dtype=np.int32)), None, None, dev(bq), dev(bs),
                             o, epdc.EPDC_FP32)
    torch.cuda.synchronize()
    got = o.double().cpu().numpy()
    want, mag = oracle.product(a, b[None], np.array([0, n]), None, None, n)
    nan = np.zeros((n, N), dtype=bool)
    nan[30], nan[:, 20] = True, True
    assert np.isnan(got[nan]).all()
    # a partial result below 2^-126 may be flushed: H of them at most
    assert np.all(np.abs(got - want)[~nan] <= ((2 * H + 4) * HALF32 * mag + H * 2.0 ** -126)[~nan])


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("experts,mean,N,H", [(65, 1, 48, 256), (130, 3, 264, 96), (200, 40, 128, 128), (300, 70, 64, 64)])
def test_expert_product_of_many_experts(experts, mean, N, H, out):
    """More experts than a wave holds at once, in each kernel."""
    rng = np.random.default_rng(experts)
    check_product(list(rng.integers(0, 2 * mean + 1, experts)), N, H, out, R=50, weighted=True, seed=experts)


@pytest.mark.parametrize("sizes", [[1, 2], [50, 60], [700, 600]])
def test_expert_product_without_rows_gives_zeros(sizes):
    n, N, H = sum(sizes), 512, 256
    bq, bs, _ = random_mx(np.random.default_rng(1), 2 * N, H)
    o = torch.full((n, N), 77.0, device="cuda")
    w = torch.full((n,), float("nan"), device="cuda")  # a row that is not there gives +0 whatever its weight
    epdc.epdc_expert_product(2, N, H, n, 0, None, None, dev(sizes_to_offsets(sizes)), None, w, dev(bq), dev(bs), o, epdc.EPDC_FP32)
    torch.cuda.synchronize()
    assert bool((o == 0).all()) and not bool(torch.signbit(o).any())


@pytest.mark.parametrize("sizes,N", [([3, 2, 0, 1], 512), ([100, 90, 120, 110, 95, 105, 99, 101], 4096), ([300] * 8, 4096)])
def test_expert_product_of_rows_beyond_32_bit_offsets(sizes, N):
    """An array of rows of 4.5 GB: the rows used lie at its start, about its 4 GB mark and at its end."""
    H, R = 8192, 1_100_000
    rng = np.random.default_rng(2)
    n, E = sum(sizes), len(sizes)
    at = np.concatenate([np.arange(20), 1_048_576 + np.arange(-10, 10), R - 1 - np.arange(20)])
    aq, as_, a = random_mx(rng, len(at), H)
    rows = torch.zeros(R, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, H // 128), 0x7F7F7F7F, dtype=torch.int32, device="cuda")
    rows[dev(at)], scales[dev(at)] = dev(aq), dev(as_)
    pick = rng.integers(0, len(at), n)
    bq, bs, b = random_mx(rng, E * N, H)
    o = torch.empty(n, N, device="cuda")
    epdc.epdc_expert_product(E, N, H, n, R, rows, scales, dev(sizes_to_offsets(sizes)), dev(at[pick].astype(np.int32)), None,
                             dev(bq), dev(bs), o, epdc.EPDC_FP32)
    torch.cuda.synchronize()
    some = np.unique(np.concatenate([np.arange(min(n, 4)), rng.integers(0, n, 20), [n - 1]]))
    expert = np.searchsorted(sizes_to_offsets(sizes), some, side="right") - 1
    b = b.reshape(E, N, H)
    for i, e in zip(some, expert):
        want, mag = b[e] @ a[pick[i]], np.abs(b[e]) @ np.abs(a[pick[i]])
        assert np.all(np.abs(o[int(i)].double().cpu().numpy() - want) <= (2 * H + 4) * HALF32 * mag), i


def test_results_and_rows_beyond_4_gb():
    """fp32 results of 4.9 GB from 300,000 entries, and quantised rows of 4.9 GB of fp32."""
    n, N, H = 300_000, 4096, 64
    rng = np.random.default_rng(3)
    aq, as_, a = random_mx(rng, 1000, H)
    bq, bs, b = random_mx(rng, N, H)
    o = torch.zeros(n, N, device="cuda")
    rows = (np.arange(n) % 1000).astype(np.int32)
    epdc.epdc_expert_product(1, N, H, n, 1000, dev(aq), dev(as_), dev(np.array([0, n], dtype=np.int32)), dev(rows), None, dev(bq),
                             dev(bs), o, epdc.EPDC_FP32)
    q = torch.empty(n, N // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(n, N // 128, dtype=torch.int32, device="cuda")
    epdc.epdc_mx_quantize(1, n, N, epdc.EPDC_FP32, o, None, q, s)
    torch.cuda.synchronize()
    for i in (0, 1, 255, 262_143, 262_144, 262_145, n - 257, n - 1):
        want, mag = b @ a[i % 1000], np.abs(b) @ np.abs(a[i % 1000])
        got = o[i].double().cpu().numpy()
        assert np.all(np.abs(got - want) <= (2 * H + 4) * HALF32 * mag), i
        want_q, want_s = oracle.pack(*oracle.mx_quantize(got[None]))
        np.testing.assert_array_equal(q[i].cpu().numpy(), want_q[0])
        np.testing.assert_array_equal(s[i].cpu().numpy(), want_s[0])
    back = torch.zeros(n, N, device="cuda")
    epdc.epdc_mx_dequantize(1, n, N, q, s, None, back, epdc.EPDC_FP32)
    torch.cuda.synchronize()
    for i in (0, 262_144, n - 1):
        want = oracle.mx_values(*oracle.unpack(q[i:i + 1].cpu().numpy(), s[i:i + 1].cpu().numpy()))
        np.testing.assert_array_equal(back[i].double().cpu().numpy(), want[0])


def test_the_same_call_twice_gives_the_same_bits():
    layer = Layer(T=100, H=512, I=256, W=4, epr=8, K=4, seed=9)
    results = []
    for _ in range(3):
        layer.out.zero_()
        layer.step()
        torch.cuda.synchronize()
        results.append([t.clone() for t in (layer.ids, layer.wts, layer.offsets, layer.of, layer.h1, layer.out)])
    for r in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], r))


# ---- streams, graphs, and all of them together --------------------------------------------------------------------


def silu_mul(x):
    n = x.shape[1] // 2
    return torch.nn.functional.silu(x[:, :n].float()) * x[:, n:].float()


class Layer:
    """A sparse feed-forward layer of T tokens: route, quantise, dispatch, group, product, activation, quantise, product,
    combine twice.  Every buffer is made once; step() only launches."""

    def __init__(self, T=48, H=256, I=128, W=4, epr=4, K=3, seed=0):
        self.T, self.H, self.I, self.W, self.epr, self.K = T, H, I, W, epr, K
        E = W * epr
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.x = rand(T, H).to(torch.bfloat16)
        self.wr = (rand(H, E) / H ** 0.5)
        self.bias = 0.05 * rand(E)
        self.w1, self.s1 = quantize((rand(E * 2 * I, H) / H ** 0.5), H, "fp32")
        self.w2, self.s2 = quantize((rand(E * H, I) / I ** 0.5), I, "fp32")
        self.rcfg = epdc.RouteCfg(E, K, epdc.EPDC_FP32, epdc.EPDC_SIGMOID, W, 2, 2, 1, 1.5)
        S = epdc.epdc_mx_scale_dim(H)
        self.dcfg = epdc.EpCfg(W, H // 2, T, epr, K, epdc.EPDC_FP4X2, 1, S)
        self.buf = epdc.DispatchBuffers(self.dcfg)
        n = self.n = W * T * K
        i32 = dict(dtype=torch.int32, device="cuda")
        self.logits = torch.zeros(T, E, device="cuda")
        self.ids, self.wts = torch.zeros(T, K, **i32), torch.zeros(T, K, device="cuda")
        self.q, self.qs = torch.zeros(T, H // 2, dtype=torch.uint8, device="cuda"), torch.zeros(T, S, device="cuda")
        self.offsets, self.row, self.of = torch.zeros(E + 1, **i32), torch.zeros(n, **i32), torch.zeros(W, T, K, **i32)
        self.ew = torch.zeros(n, device="cuda")
        self.scratch = torch.zeros(epdc.epdc_group_scratch_bytes(self.dcfg, -1) // 4, **i32)
        self.h1 = torch.zeros(n, 2 * I, dtype=torch.bfloat16, device="cuda")
        self.act = torch.zeros(n, I, device="cuda")
        self.aq = torch.zeros(n, I // 2, dtype=torch.uint8, device="cuda")
        self.aqs = torch.zeros(n, epdc.epdc_mx_scale_dim(I), **i32)
        self.h2 = torch.zeros(n, H, device="cuda")
        self.y = torch.zeros(W, T, H, device="cuda")
        self.out = torch.zeros(T, H, device="cuda")
        # the entries' rows summed into the windows' rows, then the windows' rows into the tokens
        self.c1 = epdc.EpCfg(1, H, n, max(K, 1), K, epdc.EPDC_FP32, 0, 0)
        self.c2 = epdc.EpCfg(W, H, T, epr, K, epdc.EPDC_FP32, 0, 0)

    def step(self):
        T, H, I, W, E, n, b = self.T, self.H, self.I, self.W, self.W * self.epr, self.n, self.buf
        self.logits.copy_(self.x.float() @ self.wr)
        epdc.epdc_route(self.rcfg, T, self.logits, self.bias, self.ids, self.wts)
        epdc.epdc_mx_quantize(1, T, H, epdc.EPDC_BF16, self.x, None, self.q, self.qs)
        epdc.epdc_dispatch(self.dcfg, T, self.q, self.ids, self.wts, self.qs, b.recvX, b.recvTokIdx, b.recvExpertIds,
                           b.recvWeights, b.recvScales, b.recvCount, b.sendMap, b.scratch)
        epdc.epdc_group_experts(self.dcfg, -1, b.recvExpertIds, b.recvWeights, b.recvCount, self.offsets, self.row, self.ew,
                                self.of, self.scratch)
        epdc.epdc_expert_product(E, 2 * I, H, n, W * T, b.recvX, b.recvScales, self.offsets, self.row, None, self.w1, self.s1,
                                 self.h1, epdc.EPDC_BF16)
        self.act.copy_(silu_mul(self.h1))
        epdc.epdc_mx_quantize(1, n, I, epdc.EPDC_FP32, self.act, self.offsets[E:], self.aq, self.aqs)
        epdc.epdc_expert_product(E, H, I, n, n, self.aq, self.aqs, self.offsets, None, self.ew, self.w2, self.s2, self.h2,
                                 epdc.EPDC_FP32)
        epdc.epdc_combine(self.c1, W * T, self.h2, None, None, self.of, self.y, epdc.EPDC_FP32)
        epdc.epdc_combine(self.c2, T, self.y, None, None, b.sendMap, self.out, epdc.EPDC_FP32)

    def expect(self):
        """The same layer token by token in 64 bits, from the codes that the GPU's rows must have (quantisation is
        exact, so rounding between the steps is the same on both sides but for the activations' near ties)."""
        x = self.x.double().cpu().numpy()
        l = self.logits.double().cpu().numpy()
        ids, w = oracle.route(l, self.bias.cpu().numpy(), self.K, False, self.W, 2, 2, True, 1.5)
        rows = oracle.mx_values(*oracle.mx_quantize(x))
        w1 = oracle.mx_values(*oracle.unpack(self.w1.cpu().numpy(), self.s1.cpu().numpy())).reshape(-1, 2 * self.I, self.H)
        w2 = oracle.mx_values(*oracle.unpack(self.w2.cpu().numpy(), self.s2.cpu().numpy())).reshape(-1, self.H, self.I)
        out = np.zeros_like(x)
        for t in range(self.T):
            for k in range(self.K):
                e = ids[t, k]
                if e < 0:
                    continue
                h = torch.from_numpy(rows[t] @ w1[e].T).to(torch.bfloat16).double().numpy()
                a = h[:self.I] / (1 + np.exp(-h[:self.I])) * h[self.I:]
                a = oracle.mx_values(*oracle.mx_quantize(a.astype(np.float32).astype(np.float64)[None]))[0]
                out[t] += w[t, k] * (a @ w2[e].T)
        return ids, out


def test_the_layer_together():
    layer = Layer()
    layer.step()
    torch.cuda.synchronize()
    assert epdc.dispatch_status(layer.buf.scratch) == 0
    ids, want = layer.expect()
    np.testing.assert_array_equal(layer.ids.cpu().numpy(), ids)
    got = layer.out.double().cpu().numpy()
    # An activation next to a border between two codes (or h1 next to a border of bf16) may fall to the other side:
    # a step of a code is at most a third of the value (2 to 3), on few elements.  Every token is held in the
    # 2-norm to a hundredth, 3 of 128 activations on the other side of their border.
    err = np.linalg.norm(got - want, axis=1) / np.linalg.norm(want, axis=1)
    assert np.all(err <= 0.05) and np.median(err) <= 1e-3, (err.max(), np.median(err))


def test_the_layer_in_a_graph():
    """Captured, then replayed over changed inputs with eager work between: every replay equals the eager result."""
    layer = Layer(seed=3)
    layer.step()  # eager, once before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.step()
    for seed in range(4):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(100 + seed)
        layer.x.copy_(torch.randn(layer.x.shape, device="cuda", generator=gen).to(torch.bfloat16))
        layer.out.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        replayed = layer.out.clone()
        layer.out.fill_(6.0)
        layer.step()
        torch.cuda.synchronize()
        assert torch.equal(replayed, layer.out), seed
    assert epdc.dispatch_status(layer.buf.scratch) == 0


def test_two_layers_on_two_streams():
    layers = [Layer(seed=1), Layer(T=33, H=512, I=64, K=4, seed=2)]
    alone = []
    for layer in layers:
        layer.step()
        torch.cuda.synchronize()
        alone.append(layer.out.clone())
        layer.out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for layer, s in zip(layers, streams):
            with torch.cuda.stream(s):
                layer.step()
    torch.cuda.synchronize()
    for layer, want in zip(layers, alone):
        assert torch.equal(layer.out, want)


def test_wrong_tensors_are_refused():
    c = epdc.RouteCfg(16, 2, epdc.EPDC_FP32)
    l, ids, w = torch.zeros(4, 16, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    with pytest.raises(ValueError, match="float32"):
        epdc.epdc_route(c, 4, l.bfloat16(), None, ids, w)
    with pytest.raises(ValueError, match="int32"):
        epdc.epdc_route(c, 4, l, None, ids.long(), w)
    with pytest.raises(ValueError, match="bytes"):
        epdc.epdc_route(c, 5, l, None, ids, w)
    with pytest.raises(ValueError, match="contiguous"):
        epdc.epdc_route(c, 4, torch.zeros(4, 32, device="cuda")[:, ::2], None, ids, w)
    with pytest.raises(ValueError, match="bytes"):
        epdc.epdc_mx_quantize(1, 4, 64, epdc.EPDC_FP32, torch.zeros(4, 64, device="cuda"), None,
                              torch.zeros(4, 16, dtype=torch.uint8, device="cuda"), torch.zeros(4, 1, device="cuda"))
