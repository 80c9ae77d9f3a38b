"""Routing and its gradient through each compiled form, against the 64-bit
implementation: every lane layout, kind of score and logits' type, the rounds
that blocks go when there are more tokens than one grid covers, the largest K
of the gradient's form of four tokens a wave, slots that share an expert.
tests/test_layer_ops_plans.py checks on the host which form each shape gets."""
import numpy as np
import pytest
import torch

import combine_count_amd as epdc
import layer_oracle as oracle
from test_gpu_layer_ops import HALF32, KIND, TINY, check_grad, dev, logits_of, run_grad, run_route

pytestmark = pytest.mark.gpu

# (experts, topk, groups, kept, groupTop, tokens): the form (lanes of a token, experts of a lane, in a row)
FAST = {
    (256, 8, 8, 4, 2, 150): (64, 4, 1),
    (256, 20, 16, 3, 1, 150): (64, 4, 1),
    (64, 8, 8, 4, 2, 150): (16, 4, 1),
    (64, 15, 1, 1, 1, 150): (16, 4, 1),
    (128, 6, 4, 2, 1, 150): (16, 8, 1),
    (128, 8, 1, 1, 1, 150): (16, 8, 1),
    (256, 8, 1, 1, 1, 2100): (16, 16, 1),
    (256, 8, 16, 4, 2, 2100): (16, 16, 1),
    (16, 4, 1, 1, 1, 150): (16, 4, 0),
    (50, 15, 1, 1, 1, 150): (16, 4, 0),
    (72, 6, 1, 1, 1, 150): (16, 8, 0),
    (96, 8, 1, 1, 1, 150): (16, 8, 0),
    (160, 6, 1, 1, 1, 150): (16, 16, 0),
    (192, 8, 1, 1, 1, 150): (16, 16, 0),
    (250, 15, 1, 1, 1, 150): (16, 16, 0),
    (100, 20, 1, 1, 1, 150): (64, 4, 0),
    (256, 16, 1, 1, 1, 2100): (64, 4, 0),
    (384, 8, 1, 1, 1, 150): (64, 8, 0),
    (1000, 63, 1, 1, 1, 60): (64, 16, 0),
}
# the general form: a softmax with a bias, groups that are no whole lanes, as many choices as lanes
GENERAL = {
    (60, 4, 4, 2, 2, 150): (0, 1, 0),
    (120, 8, 6, 3, 1, 150): (0, 2, 0),
    (160, 8, 8, 3, 2, 150): (0, 4, 0),
    (512, 10, 16, 4, 1, 60): (0, 8, 0),
    (1024, 64, 64, 32, 2, 40): (0, 16, 0),
}
SCORES = [("sigmoid", False), ("softmax", True), ("softmax", False)]  # (score, renormalised)


def is_biased(form, score):
    """A sigmoid has a bias; a softmax has one in the general form."""
    return score == "sigmoid" or form in GENERAL


def route_shapes():
    """(E, K, G, keep, T, softmax, biased, aligned): form, of every call of test_every_form."""
    return {(E, K, G, keep, T, int(score == "softmax"), int(is_biased(c, score)), 1): {**FAST, **GENERAL}[c]
            for c in (*FAST, *GENERAL) for E, K, G, keep, _, T in [c] for score, _ in SCORES}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score,renorm", SCORES)
@pytest.mark.parametrize("cfg", [*FAST, *GENERAL], ids=lambda c: "-".join(map(str, c)))
def test_every_form(cfg, score, renorm, dtype):
    E, K, G, keep, top, T = cfg
    rng = np.random.default_rng(E * 100 + K)
    # a fifth of the tokens each: ordinary, nearly equal, masked, ties, far apart
    parts = []
    for i, values in enumerate(("normal", "near", "masked", "ties", "wide")):
        n = -(-T // 5) if i < 4 else T - 4 * -(-T // 5)
        if values == "near":
            parts.append(rng.standard_normal((n, 1)) + rng.integers(-3, 4, (n, E)) * 2.0 ** -22)
        else:
            parts.append(logits_of(values, n, E, dtype, rng)[1])
    l = np.concatenate(parts)[rng.permutation(T)]
    t = torch.from_numpy(l).to(KIND[dtype][1])
    l = t.double().numpy()
    bias = (0.2 * rng.standard_normal(E)).astype(np.float32) if is_biased(cfg, score) else None
    ids, w = run_route(E, K, G, keep, top, score, renorm, 2.5, dtype, t.cuda(), None if bias is None else dev(bias))
    want_ids, want = oracle.route(l, bias, K, score == "softmax", G, keep, top, renorm, 2.5)
    np.testing.assert_array_equal(ids, want_ids)
    # computed in 64 bits and rounded once: half a step, and what 64 bits are off themselves
    assert np.all(np.abs(w - want) <= HALF32 * (1 + 2.0 ** -20) * np.abs(want) + TINY["fp32"])


GRID = 1 << 20  # the most blocks of a launch; a block takes 4 tokens, or 16 where a wave takes four

# (tokens of a block, experts, topk, groups, kept, groupTop, score, bias)
ROUNDS = [(16, 8, 2, 1, 1, 1, "sigmoid", True), (16, 64, 6, 8, 4, 2, "sigmoid", True), (4, 16, 16, 1, 1, 1, "softmax", False),
          (4, 8, 2, 4, 2, 2, "softmax", True)]


def round_shapes():
    form = {16: 16, 4: 64}
    return {(E, K, G, keep, per * GRID + 777, int(score == "softmax"), int(biased), 1):
            0 if score == "softmax" and biased else form[per] for per, E, K, G, keep, _, score, biased in ROUNDS}


def some_tokens(first, T, rng):
    """Of the first round's start and end, and of the second round."""
    return np.unique(np.concatenate([np.arange(8), first - 1 - np.arange(8), first + np.arange(T - first),
                                     rng.integers(0, first, 30)]))


@pytest.mark.parametrize("per,E,K,G,keep,top,score,biased", ROUNDS)
def test_more_tokens_than_one_grid(per, E, K, G, keep, top, score, biased):
    first = per * GRID
    T = first + 777
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    l = torch.randint(-24, 24, (T, E), device="cuda", generator=g, dtype=torch.int16).to(torch.bfloat16) / 8  # with ties
    bias = 0.1 * torch.randn(E, device="cuda", generator=g) if biased else None
    cfg = epdc.RouteCfg(E, K, epdc.EPDC_BF16, epdc.EPDC_SOFTMAX if score == "softmax" else epdc.EPDC_SIGMOID, G, keep, top, 1, 1.0)
    ids = torch.full((T + 1, K), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, K), -7.0, device="cuda")
    epdc.epdc_route(cfg, T, l, bias, ids, w)
    part_ids, part_w = torch.empty_like(ids[:T]), torch.empty_like(w[:T])
    for t0 in range(0, T, first // 2):  # in calls of one round each
        n = min(first // 2, T - t0)
        epdc.epdc_route(cfg, n, l[t0:t0 + n], bias, part_ids[t0:t0 + n], part_w[t0:t0 + n])
    torch.cuda.synchronize()
    assert bool((ids[T] == -77).all()) and bool((w[T] == -7.0).all())
    assert torch.equal(ids[:T], part_ids) and torch.equal(w[:T], part_w)
    at = some_tokens(first, T, np.random.default_rng(E))
    x = l[dev(at)].double().cpu().numpy()
    want_ids, want = oracle.route(x, None if bias is None else bias.cpu().numpy(), K, score == "softmax", G, keep, top, True, 1.0)
    np.testing.assert_array_equal(ids[dev(at)].cpu().numpy(), want_ids)
    assert np.all(np.abs(w[dev(at)].double().cpu().numpy() - want) <= HALF32 * (1 + 2.0 ** -20) * want)


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("per,E,K", [(4, 8, 2), (16, 64, 6)])
def test_more_tokens_than_one_grid_in_the_gradient(per, E, K, score, renorm):
    first = per * GRID
    T = first + 777
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    l = torch.randint(-24, 24, (T, E), device="cuda", generator=g, dtype=torch.int16).to(torch.bfloat16) / 8
    ids = torch.randint(-1, E, (T, K), device="cuda", generator=g, dtype=torch.int32)
    dw = torch.randn(T, K, device="cuda", generator=g)
    cfg = epdc.RouteCfg(E, K, epdc.EPDC_BF16, epdc.EPDC_SOFTMAX if score == "softmax" else epdc.EPDC_SIGMOID, 1, 1, 1, int(renorm), 1.0)
    d = torch.full((T + 1, E), 9.0, dtype=torch.bfloat16, device="cuda")
    epdc.epdc_route_grad(cfg, T, l, ids, dw, d)
    part = torch.empty_like(d[:T])
    for t0 in range(0, T, first // 2):
        n = min(first // 2, T - t0)
        epdc.epdc_route_grad(cfg, n, l[t0:t0 + n], ids[t0:t0 + n], dw[t0:t0 + n], part[t0:t0 + n])
    torch.cuda.synchronize()
    assert bool((d[T] == 9.0).all())
    assert torch.equal(d[:T], part)
    at = dev(some_tokens(first, T, np.random.default_rng(E)))
    check_grad(d[at].double().cpu().numpy(), l[at].double().cpu().numpy(), ids[at].cpu().numpy(), dw[at].cpu().numpy(), score, renorm,
               1.0, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [64, 128, 256])
@pytest.mark.parametrize("K", [15, 16, 17])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_gradient_around_sixteen_slots(score, renorm, K, E, dtype):
    """Up to 16 slots: four tokens a wave, a slot in each of a token's lanes; from 17 a token a wave."""
    rng = np.random.default_rng(E + K)
    t, l = logits_of("normal", 45, E, dtype, rng)
    ids = oracle.route(l, None, K, score == "softmax")[0]
    ids[rng.random(ids.shape) < 0.1] = -1
    dw = rng.standard_normal((45, K)).astype(np.float32)
    check_grad(run_grad(E, K, score, renorm, 2.5, dtype, t.cuda(), ids, dw), l, ids, dw, score, renorm, 2.5, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [64, 96, 128, 256])
@pytest.mark.parametrize("K", [6, 16])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_gradient_of_slots_that_share_an_expert(score, renorm, K, E, dtype):
    rng = np.random.default_rng(E + K)
    T = 37
    t, l = logits_of("normal", T, E, dtype, rng)
    ids = rng.integers(E - 4, E, (T, K)).astype(np.int32)
    ids[0], ids[1, 1:] = E - 1, -1  # all slots one expert; one slot alone
    dw = rng.standard_normal((T, K)).astype(np.float32)
    check_grad(run_grad(E, K, score, renorm, 1.5, dtype, t.cuda(), ids, dw), l, ids, dw, score, renorm, 1.5, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [96, 128])
@pytest.mark.parametrize("above", [float("inf"), 900.0])
def test_softmax_shares_of_scores_that_vanish(above, E, dtype):
    """An expert that its bias masks has a logit so far above all others that the chosen scores vanish in 64 bits: the
    weights are 0, the gradient is that of the shares among the slots (include/epdc.h)."""
    rng = np.random.default_rng(E)
    T, K, scale = 21, 5, 2.0
    l = rng.standard_normal((T, E))
    l[:, 7] = above
    t = torch.from_numpy(l).to(KIND[dtype][1])
    l = t.double().numpy()
    bias = np.zeros(E, dtype=np.float32)
    bias[7] = -np.inf
    bias[10:20] = 0.5
    ids, w = run_route(E, K, 1, 1, 1, "softmax", True, scale, dtype, t.cuda(), dev(bias))
    assert not w.any() and (ids == np.arange(10, 10 + K)).all()  # choice values all 0.5: the lowest of them
    dw = rng.standard_normal((T, K)).astype(np.float32)
    check_grad(run_grad(E, K, "softmax", True, scale, dtype, t.cuda(), ids, dw), l, ids, dw, "softmax", True, scale, dtype)
    # no slot, no gradient; nor without a gradient of the weights
    assert not run_grad(E, K, "softmax", True, scale, dtype, t.cuda(), np.full_like(ids, -1), dw).any()
    assert not run_grad(E, K, "softmax", True, scale, dtype, t.cuda(), ids, np.zeros_like(dw)).any()
