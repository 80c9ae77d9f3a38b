"""Routing through each compiled form, against the 64-bit implementation:
every lane layout, kind of score and logits' type.  tests/test_layer_ops_plans.py
checks on the host which form each shape gets."""
import numpy as np
import pytest
import torch

import layer_oracle as oracle
from test_gpu_layer_ops import HALF32, KIND, TINY, dev, logits_of, run_route

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
