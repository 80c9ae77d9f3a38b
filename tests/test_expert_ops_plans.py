"""Which kernel the experts' products in bf16 and int8 run for a shape (host
code of csrc/ops_internal.h that the launchers run): the shapes the rule was
measured on, and that the GPU tests reach every compiled form, so that a changed
rule cannot move the tests away from a kernel unseen."""
import os
import subprocess

import pytest

from combine_count_amd import _build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FORMS = ("stream16", "stream64", "tiles128", "tiles256")
PRODUCT, ROWS, WEIGHTS = 0, 1, 2


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plans") / "expert_plan_check")
    src = os.path.join(ROOT, "tests", "host", "expert_plan_check.cpp")
    r = subprocess.run([B.HIPCC, *B.COMMON, src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(shapes):
        r = subprocess.run([exe, *[str(v) for s in shapes for v in s]], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        rows = [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
        return {row[:5]: FORMS[row[5]] for row in rows}

    return run


# (kind, experts, columns, hidden, maxEntries): form
EXPECT = {
    # few entries, and tiles of 128 would leave CUs idle
    (PRODUCT, 1, 4096, 7168, 1): "stream16",
    (PRODUCT, 1, 4096, 7168, 16): "stream16",
    (PRODUCT, 1, 4096, 7168, 64): "stream64",
    (PRODUCT, 2, 4096, 7168, 64): "stream64",
    (PRODUCT, 4, 4096, 7168, 128): "stream64",
    (PRODUCT, 8, 4096, 7168, 64): "stream16",
    (PRODUCT, 8, 4096, 7168, 256): "tiles128",
    (PRODUCT, 1, 4096, 7168, 256): "stream64",
    (PRODUCT, 1, 4096, 7168, 512): "tiles128",
    (PRODUCT, 32, 4096, 7168, 64): "tiles128",
    # the mean group fills a good part of a 256-row tile, and there is one for every CU
    (PRODUCT, 8, 4096, 7168, 2048): "tiles128",
    (PRODUCT, 8, 4096, 7168, 4096): "tiles256",
    (PRODUCT, 32, 4096, 7168, 4096): "tiles128",
    (PRODUCT, 32, 7168, 2048, 8192): "tiles256",
    (PRODUCT, 1, 4096, 7168, 8192): "tiles256",
    (PRODUCT, 32, 7168, 2048, 2047): "tiles128",
    (PRODUCT, 32, 4096, 7168, 32768): "tiles256",
    (ROWS, 8, 520, 1000, 777): "tiles128",
    (ROWS, 32, 7168, 2048, 16384): "tiles256",
    (WEIGHTS, 16, 1024, 1000, 333): "tiles256",
    (WEIGHTS, 32, 4096, 7168, 16384): "tiles256",
    (WEIGHTS, 2, 136, 264, 100): "tiles128",
}


def test_forms(plan):
    assert plan(list(EXPECT)) == EXPECT


def test_the_gpu_tests_reach_every_form(plan):
    import test_gpu_expert_forms as F
    shapes = F.product_shapes()
    got = plan([s[1:] for s in shapes])
    assert all(got[s[1:]] == s[0] for s in shapes)
    import test_gpu_expert_ops as T
    for kind in (PRODUCT, ROWS, WEIGHTS):
        small = [(kind, len(sizes), N, H, sum(sizes) + first + behind) for sizes, first, behind in T.GROUPS.values()
                 for N, H in T.SHAPES]
        # ninety experts of larger weights are tiles enough for the next form
        want = {PRODUCT: {"stream16", "stream64", "tiles128"}, ROWS: {"tiles128"}, WEIGHTS: {"tiles128", "tiles256"}}
        assert set(plan(small).values()) == want[kind]


def test_the_streamed_shapes_reach_their_forms(plan):
    import test_gpu_expert_stream as F
    shapes = F.shapes()
    got = plan([s[1:] for s in shapes])
    assert all(got[s[1:]] == s[0] for s in shapes)


def test_the_shapes_of_many_tiles_reach_the_tiles_of_128(plan):
    import test_gpu_expert_many_tiles as F
    shapes = F.shapes()
    got = plan([s[1:] for s in shapes])
    assert all(got[s[1:]] == s[0] for s in shapes)
    assert F.tiles() > 2.5 * F.BLOCKS
