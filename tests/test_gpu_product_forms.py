"""The experts' product through each of its LDS-tile kernels, against the
64-bit implementation: every number of steps and every ending of the rows,
both types of results, groups that end inside a tile, more tiles than blocks
that run at once, missing rows, offsets that run backwards, NaN scales.

The kernel follows from maxEntries, which may exceed the entries there are:
each form's shapes pass a capacity that selects it, whatever the groups hold
(tests/test_layer_ops_plans.py checks on the host that they do)."""
import numpy as np
import pytest
import torch

import combine_count_amd as epdc
import layer_oracle as oracle
from test_gpu_layer_ops import HALF, HALF32, KIND, dev, random_mx, sizes_to_offsets

pytestmark = pytest.mark.gpu

WIDE_BYTES = 4_500_000_000  # an array of rows whose offsets pass 32 bits
# form: (columns of the small cases, capacity of the small cases)
FORMS = {"tiles128": (136, 20000), "tiles128_wide": (136, 20000), "tiles256": (520, 44000)}
SMALL = [47, 300, 0, 131]  # ends inside a tile of each height
HIDDEN = [256 * steps - tail for steps in range(1, 12) for tail in (0, 32, 128, 224)]


def sizes_of(E, largest, seed):
    return list(np.random.default_rng(seed).integers(0, largest + 1, E))


# (form, columns, hidden, groups' sizes): more tiles than the 512 or 256 blocks that run at once, so that blocks go on
# to a second and a third tile; more experts than a wave holds at once
MANY = [(form, N, H, E, largest) for form, N, E, largest in
        (("tiles128", 1032, 70, 260), ("tiles128_wide", 1032, 70, 260), ("tiles256", 1032, 70, 600))
        for H in (96, 416, 736, 1024, 1184)]


def rows_of(form, n, H):
    """Rows in the array: as many as there are entries' rows, or enough to pass 32-bit offsets."""
    return WIDE_BYTES // (H // 2) if form == "tiles128_wide" else max(n, 1)


def shapes():
    """(form, E, N, H, maxEntries, numRows) of every call below."""
    out = []
    for form, (N, cap) in FORMS.items():
        for H in HIDDEN:
            out.append((form, len(SMALL), N, H, cap, rows_of(form, 97, H)))
    for form, N, H, E, largest in MANY:
        n = sum(sizes_of(E, largest, H))
        out.append((form, E, N, H, n, rows_of(form, 97, H)))
    return out


@pytest.fixture(scope="module")
def wide():
    """4.5 GB for rows, and for their scales (of rows of 32 elements, the most scale bytes for their size)."""
    yield torch.zeros(WIDE_BYTES, dtype=torch.uint8, device="cuda"), torch.full((WIDE_BYTES // 16,), 0x7F7F7F7F,
                                                                               dtype=torch.int32, device="cuda")
    torch.cuda.empty_cache()


def check(form, sizes, N, H, out, cap, wide, seed, offsets=None, missing=False, nan=False):
    rng = np.random.default_rng(seed)
    E = len(sizes)
    offsets = sizes_to_offsets(sizes) if offsets is None else np.asarray(offsets, dtype=np.int32)
    n = min(int(offsets.max()), cap)
    R, some = rows_of(form, 97, H), 97
    aq, as_, a = random_mx(rng, some, H)
    bq, bs, b = random_mx(rng, E * N, H)
    nan_row, nan_col = (5, 7) if nan else (-1, -1)
    if nan:  # one block of one row and of one column of every expert
        block = H // 32 - 1
        as_.view(np.uint8).reshape(some, -1)[nan_row, block] = 255
        bs.view(np.uint8).reshape(E, N, -1)[:, nan_col, block] = 255
    if form == "tiles128_wide":  # the rows used: at the start, about the 4 GB mark, at the end
        mark = 2 ** 32 // (H // 2)
        at = np.concatenate([np.arange(33), mark - 16 + np.arange(32), R - 32 + np.arange(32)])
        rows_d = wide[0][:R * (H // 2)].view(R, H // 2)
        words = epdc.epdc_mx_scale_dim(H)
        scales_d = wide[1][:R * words].view(R, words)
        rows_d[dev(at)], scales_d[dev(at)] = dev(aq), dev(as_)
    else:
        at, rows_d, scales_d = np.arange(some), dev(aq), dev(as_)
    pick = rng.integers(0, some, n)
    rows = at[pick].astype(np.int32)
    w = rng.standard_normal(n).astype(np.float32)
    if missing:
        rows[::5] = np.resize(np.array([-1, R, 2 ** 31 - 1, -2 ** 31], dtype=np.int32), len(rows[::5]))
        w[::10] = np.nan  # a row that is not there gives +0 whatever its weight
        pick[::5] = -1
    full_rows, full_w = np.full(cap, -1, dtype=np.int32), np.zeros(cap, dtype=np.float32)
    full_rows[:n], full_w[:n] = rows, w
    o = torch.full((cap, N), 77.0, dtype=KIND[out][1], device="cuda")
    epdc.epdc_expert_product(E, N, H, cap, R if form == "tiles128_wide" else some, rows_d, scales_d, dev(offsets), dev(full_rows),
                             dev(full_w), dev(bq), dev(bs), o, KIND[out][0])
    torch.cuda.synchronize()
    assert bool((o[n:] == 77.0).all())  # nothing behind the last group
    got = o[:n].double().cpu().numpy()
    want, mag = oracle.product(a, b.reshape(E, N, H), offsets, pick, np.where(pick < 0, 0, w), n)
    none = np.isnan(want)  # entries of no group
    assert (got[none] == 77.0).all()
    poisoned = np.zeros_like(none)
    if nan:
        poisoned[pick == nan_row] = True
        poisoned[:, nan_col] = True
        poisoned[pick < 0] = False
        poisoned &= ~none
        assert np.isnan(got[poisoned]).all()
    if missing:
        gone = (pick < 0)[:, None] & ~none
        assert (got[gone] == 0).all() and not np.signbit(got[gone]).any()
    # H products exact in 32 bits, H additions in any order, the weight; a truncating addition is off by a whole
    # step: two half steps each; then the result's rounding
    bound = (2 * H + 4) * HALF32 * mag + HALF[out] * np.abs(want)
    bad = ~none & ~poisoned & ~(np.abs(got - want) <= bound)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("H", HIDDEN)
@pytest.mark.parametrize("form", FORMS)
def test_every_number_of_steps(form, H, out, wide):
    N, cap = FORMS[form]
    check(form, SMALL, N, H, out, cap, wide, seed=H)


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("form,N,H,E,largest", MANY)
def test_more_tiles_than_blocks(form, N, H, E, largest, out, wide):
    sizes = sizes_of(E, largest, H)
    height = 256 if form == "tiles256" else 128
    assert sum(-(-s // height) for s in sizes) * -(-N // height) > (256 if form == "tiles256" else 512)
    check(form, sizes, N, H, out, sum(sizes), wide, seed=H + 1)


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [160, 512, 1376])
@pytest.mark.parametrize("form", FORMS)
def test_missing_rows_and_backward_offsets(form, H, out, wide):
    N, cap = FORMS[form]
    # entries before the first group; a group that runs backwards is empty, the one in front of it ends where that begins
    check(form, SMALL, N, H, out, cap, wide, seed=H, offsets=[3, 300, 170, 170, 441], missing=True)


@pytest.mark.parametrize("form", FORMS)
def test_offsets_beyond_the_capacity(form, wide):
    N, cap = FORMS[form]
    check(form, SMALL, N, 32, "fp32", cap, wide, seed=1, offsets=[-5, 40, cap - 30, 2 ** 31 - 1, 2 ** 31 - 1])


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [96, 512, 736, 1056])
@pytest.mark.parametrize("form", FORMS)
def test_nan_scales_reach_their_row_and_column_alone(form, H, out, wide):
    N, cap = FORMS[form]
    check(form, SMALL, N, H, out, cap, wide, seed=H, missing=True, nan=True)
