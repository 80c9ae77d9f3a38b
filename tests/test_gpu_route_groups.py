"""The choice of groups where a group's score is a small sum of large terms:
biases of both signs in one group.  The 32-bit form of the router has to see
that its sums cannot tell such groups apart, whatever the sums' own size."""
import numpy as np
import pytest
import torch

import combine_count_amd as epdc
import layer_oracle as oracle

pytestmark = pytest.mark.gpu

KIND = {"bf16": (epdc.EPDC_BF16, torch.bfloat16), "fp32": (epdc.EPDC_FP32, torch.float32)}


def biases(kind, E, G, rng):
    """[E] fp32.  1e4, 1e6: one expert of each group raised by as much and the others lowered; pinned: one expert out of
    reach upwards in a group whose others are switched off with a finite number, beside ordinary groups; infinite: an
    expert of most groups at +inf, its neighbours far below."""
    per = E // G
    b = (0.1 * rng.standard_normal(E)).astype(np.float32)
    if kind == "pinned":
        b[per:2 * per] = -1e9
        b[per + 3] = 1e9
    elif kind == "infinite":
        b[1::per] = -3e38
        b[:5 * per:per] = np.inf
    else:
        b[:] = -float(kind)
        b[::per] = float(kind)
    return b


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["1e4", "1e6", "pinned", "infinite"])
@pytest.mark.parametrize("E,T", [(256, 2000), (256, 3000), (128, 3000), (64, 3000)])
def test_groups_whose_terms_cancel(E, T, kind, dtype):
    G, keep, K = 8, 4, 8
    rng = np.random.default_rng(E + T)
    t = torch.from_numpy(rng.standard_normal((T, E))).to(KIND[dtype][1])
    bias = biases(kind, E, G, rng)
    cfg = epdc.RouteCfg(E, K, KIND[dtype][0], epdc.EPDC_SIGMOID, G, keep, 2, 1, 2.5)
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    epdc.epdc_route(cfg, T, t.cuda(), torch.from_numpy(bias).cuda(), ids, w)
    torch.cuda.synchronize()
    want_ids, want = oracle.route(t.double().numpy(), bias, K, False, G, keep, 2, True, 2.5)
    wrong = (ids.cpu().numpy() != want_ids).any(1)
    assert not wrong.any(), f"{wrong.sum()} of {T} tokens, first {np.flatnonzero(wrong)[:5]}"
    # computed in 64 bits and rounded once
    assert np.all(np.abs(w.double().cpu().numpy() - want) <= 2.0 ** -24 * (1 + 2.0 ** -20) * want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [500, 2500])
def test_groups_of_scores_near_nothing(T, score):
    """One expert far above all others, two-best groups without a bias: the groups left over differ in scores far below
    what 32-bit sums resolve."""
    rng = np.random.default_rng(T)
    E, G, keep, K = 256, 8, 4, 8
    l = (3.0 * rng.standard_normal((T, E)) - 60.0).astype(np.float32)
    l[np.arange(T), rng.integers(0, E, T)] = 5.0
    cfg = epdc.RouteCfg(E, K, epdc.EPDC_FP32, epdc.EPDC_SOFTMAX if score == "softmax" else epdc.EPDC_SIGMOID, G, keep, 2, 1, 1.0)
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    epdc.epdc_route(cfg, T, torch.from_numpy(l).cuda(), None, ids, w)
    torch.cuda.synchronize()
    want_ids, want = oracle.route(l, None, K, score == "softmax", G, keep, 2, True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    assert np.all(np.abs(w.double().cpu().numpy() - want) <= 2.0 ** -24 * (1 + 2.0 ** -20) * want + 2.0 ** -150)
