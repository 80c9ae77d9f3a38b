"""Which kernel the operators next to dispatch and combine run for a shape
(host code of csrc/ops_internal.h that the launchers run): the shapes the
rules were measured on, and that the GPU tests reach every compiled form, so
that a changed rule cannot move the tests away from a kernel unseen."""
import os
import subprocess

import pytest

from combine_count_amd import _build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PRODUCT = ("stream16", "stream64", "tiles128", "tiles128_wide", "tiles256")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plans") / "layer_plan_check")
    src = os.path.join(ROOT, "tests", "host", "layer_plan_check.cpp")
    r = subprocess.run([B.HIPCC, *B.COMMON, src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(kind, shapes):
        r = subprocess.run([exe, kind, *[str(v) for s in shapes for v in s]], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        rows = [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
        return {row[:len(shapes[0])]: row[len(shapes[0]):] for row in rows}

    return run


# (experts, columns, hidden, maxEntries, rows): form
PRODUCT_EXPECT = {
    # a few entries of each expert, long rows
    (32, 4096, 7168, 64, 8): "stream16",
    (32, 4096, 7168, 128, 16): "stream16",
    (32, 4096, 7168, 129, 17): "tiles128",
    (32, 4096, 4096, 64, 8): "tiles128",
    # 128 x 128 tiles would leave CUs idle
    (1, 4096, 7168, 8, 8): "stream16",
    (8, 4096, 7168, 8, 8): "stream16",
    (2, 4096, 7168, 64, 64): "stream64",
    (8, 4096, 7168, 128, 128): "tiles128",
    # uneven groups, second product of an expert
    (32, 7168, 2048, 2047, 2047): "tiles128",
    # the mean group fills a good part of a 256-row tile, and there are two rounds of them
    (32, 4096, 7168, 3000, 3000): "tiles128",
    (32, 4096, 7168, 4096, 4096): "tiles256",
    (32, 4096, 7168, 32768, 16384): "tiles256",
    # rows past 32-bit offsets
    (32, 4096, 7168, 32768, 1123474): "tiles256",
    (32, 4096, 7168, 32768, 1123475): "tiles128_wide",
}


def test_product_forms(plan):
    got = plan("product", list(PRODUCT_EXPECT))
    assert {k: PRODUCT[v[0]] for k, v in got.items()} == PRODUCT_EXPECT


def test_the_gpu_tests_reach_every_product_form(plan):
    import test_gpu_product_forms as F
    shapes = F.shapes()
    got = plan("product", [s[1:] for s in shapes])
    assert [PRODUCT[got[s[1:]][0]] for s in shapes] == [s[0] for s in shapes]
    assert {s[0] for s in shapes} == set(PRODUCT) - {"stream16", "stream64"}


def test_the_step_tests_of_small_groups_run_the_streaming_kernels(plan):
    """The shapes of test_gpu_layer_ops.test_expert_product_every_number_of_steps: the other two forms."""
    shapes = [(2, 136, 256 * steps - tail, rows + rows + 7, 97) for steps in range(1, 12) for tail in (0, 32, 128, 224)
              for rows in (40, 300)]
    assert {PRODUCT[v[0]] for v in plan("product", shapes).values()} == {"stream64"}
    shapes = [(8, 2048, 7168, 11, 8), (3, 8, 64, 6, 5), (40, 264, 1056, 83, 16)]  # of test_expert_product
    assert {PRODUCT[v[0]] for v in plan("product", shapes).values()} == {"stream16"}


def test_the_gpu_tests_reach_every_routing_form(plan):
    import test_gpu_route_forms as F
    want = F.route_shapes()
    assert plan("route", list(want)) == want
    compiled = {(64, 4, 1)} | {(16, n, r) for n in (4, 8, 16) for r in (0, 1)} | {(64, n, 0) for n in (4, 8, 16)}
    compiled |= {(0, n, 0) for n in (1, 2, 4, 8, 16)}
    for softmax in (0, 1):  # of either score
        assert {v for k, v in want.items() if k[5] == softmax} == compiled
    rounds = F.round_shapes()
    assert {k: v[0] for k, v in plan("route", list(rounds)).items()} == rounds


def test_gradient_forms(plan):
    expect = {(64, 16, 1): (16, 4, 1), (128, 16, 1): (16, 8, 1), (256, 16, 1): (16, 16, 1), (64, 17, 1): (0, 1, 0),
              (128, 17, 1): (0, 2, 0), (256, 17, 1): (0, 4, 0), (256, 8, 0): (0, 4, 0), (96, 6, 1): (0, 2, 0), (384, 8, 1): (0, 8, 0),
              (1024, 9, 1): (0, 16, 0), (8, 2, 1): (0, 1, 0)}
    assert plan("grad", list(expect)) == expect


# (experts, topk, groups, kept, tokens, softmax, bias, aligned): (lanes, experts of a lane, in a row)
ROUTE_EXPECT = {
    (256, 8, 8, 4, 2048, 0, 1, 1): (64, 4, 1),
    (256, 8, 8, 4, 2049, 0, 1, 1): (16, 16, 1),
    (256, 8, 8, 4, 2049, 0, 1, 0): (0, 4, 0),  # groups of logits between 16-byte borders
    (256, 8, 1, 1, 2049, 0, 1, 0): (16, 16, 0),
    (256, 8, 1, 1, 4096, 1, 0, 1): (16, 16, 1),
    (256, 8, 1, 1, 4096, 1, 1, 1): (0, 4, 0),  # a softmax with a bias
    (160, 6, 8, 3, 4096, 1, 0, 1): (0, 4, 0),  # groups of 20
    (160, 6, 8, 8, 4096, 1, 0, 1): (16, 16, 0),  # no limit
}


def test_route_forms(plan):
    assert plan("route", list(ROUTE_EXPECT)) == ROUTE_EXPECT
