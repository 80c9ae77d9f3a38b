"""Host checks of the operators next to dispatch and combine: every refusal
with its documented code before anything is launched, and the binding's own
checks of its tensors.  No GPU is needed."""
import math
import os
import re

import pytest
import torch

import combine_count_amd as epdc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P16 = 0x10000  # a fake, 16-byte aligned device address: never dereferenced on these paths

ROUTE = dict(numExperts=256, numExpertPerToken=8, dtype=0, score=1, numGroups=8, groupsPerToken=4, groupTop=2,
             renormalize=1, routedScale=2.5)
CFG = dict(worldSize=8, hiddenDim=7168, maxTokPerRank=4096, numExpertPerRank=32, numExpertPerToken=8, dtype=0,
           useWeights=1, scaleDim=0)


def test_header_constants():
    src = open(os.path.join(ROOT, "include", "epdc.h")).read()
    for name in ("EPDC_SOFTMAX", "EPDC_SIGMOID", "EPDC_MAX_ROUTE_EXPERTS", "EPDC_MAX_GROUP_EXPERTS"):
        v = re.search(rf"{name}\s*(?:=\s*)?(\d+)", src)
        assert v and int(v.group(1)) == getattr(epdc, name), name


def test_scale_dim():
    assert [epdc.epdc_mx_scale_dim(c) for c in (32, 128, 160, 7168, 128 * 1024)] == [1, 1, 2, 56, 1024]
    assert [epdc.epdc_mx_scale_dim(c) for c in (0, -32, 16, 100, 128 * 1024 + 32)] == [-1] * 5


ROUTE_REJECT = [
    ("no experts", dict(numExperts=0, numGroups=1), 8, {}, -1),
    ("too many experts", dict(numExperts=1025, numGroups=1, groupsPerToken=1), 8, {}, -1),
    ("topk 0", dict(numExpertPerToken=0), 8, {}, -1),
    ("topk 65", dict(numExpertPerToken=65), 8, {}, -1),
    ("topk beyond the kept groups", dict(numExpertPerToken=33, groupsPerToken=1), 8, {}, -1),
    ("topk beyond the experts", dict(numExperts=4, numGroups=1, groupsPerToken=1), 8, {}, -1),
    ("groups do not divide", dict(numGroups=7), 8, {}, -1),
    ("65 groups", dict(numExperts=650, numGroups=65), 8, {}, -1),
    ("no group kept", dict(groupsPerToken=0), 8, {}, -1),
    ("more groups kept than there are", dict(groupsPerToken=9), 8, {}, -1),
    ("groupTop 0", dict(groupTop=0), 8, {}, -1),
    ("groupTop 3", dict(groupTop=3), 8, {}, -1),
    ("groupTop above a group's experts", dict(numExperts=8, numGroups=8, groupsPerToken=8), 8, {}, -1),
    ("scale not finite", dict(routedScale=math.inf), 8, {}, -1),
    ("scale NaN", dict(routedScale=math.nan), 8, {}, -1),
    ("negative tokens", {}, -1, {}, -1),
    ("dtype fp8", dict(dtype=2), 8, {}, -2),
    ("score 2", dict(score=2), 8, {}, -2),
    ("renormalize 2", dict(renormalize=2), 8, {}, -2),
    ("logits odd address", {}, 8, dict(logits=P16 + 1), -4),
    ("fp32 logits at 2 bytes", dict(dtype=1), 8, dict(logits=P16 + 2), -4),
    ("ids misaligned", {}, 8, dict(ids=P16 + 2), -4),
    ("weights misaligned", {}, 8, dict(w=P16 + 1), -4),
    ("logits null", {}, 8, dict(logits=None), -5),
    ("ids null", {}, 8, dict(ids=None), -5),
    ("weights null", {}, 8, dict(w=None), -5),
]


@pytest.mark.parametrize("what,over,T,ptrs,code", ROUTE_REJECT, ids=[r[0] for r in ROUTE_REJECT])
def test_route_and_its_gradient_reject(what, over, T, ptrs, code):
    c = epdc.RouteCfg(**{**ROUTE, **over})
    a = dict(logits=P16, ids=P16, w=P16)
    a.update(ptrs)
    assert epdc.epdc_route(c, T, a["logits"], P16, a["ids"], a["w"], stream=0, check=False) == code
    assert epdc.epdc_last_error() != ""
    assert epdc.epdc_route_grad(c, T, a["logits"], a["ids"], a["w"], P16, stream=0, check=False) == code
    assert epdc.epdc_last_error() != ""


def test_route_rejects_its_own():
    c = epdc.RouteCfg(**ROUTE)
    assert epdc.epdc_route(c, 8, P16, P16 + 2, P16, P16, stream=0, check=False) == -4  # bias
    assert epdc.epdc_route_grad(c, 8, P16, P16, P16, None, stream=0, check=False) == -5
    assert epdc.epdc_route_grad(c, 8, P16, P16, P16, P16 + 1, stream=0, check=False) == -4
    # no tokens: nothing to do, nothing needed
    assert epdc.epdc_route(c, 0, None, None, None, None, stream=0) == 0
    assert epdc.epdc_route_grad(c, 0, None, None, None, None, stream=0) == 0


MX_REJECT = [
    ("negative windows", dict(W=-1), -1),
    ("negative rows", dict(M=-1), -1),
    ("too many rows", dict(W=1 << 16, M=1 << 15), -1),
    ("cols 0", dict(cols=0), -1),
    ("cols 48", dict(cols=48), -1),
    ("cols beyond the scale limit", dict(cols=128 * 1024 + 32), -1),
    ("dtype fp4x2", dict(dtype=3), -2),
    ("dtype fp8", dict(dtype=2), -2),
    ("rows misaligned", dict(x=P16 + 8), -4),
    ("q misaligned", dict(q=P16 + 4), -4),
    ("scales misaligned", dict(s=P16 + 2), -4),
    ("count misaligned", dict(count=P16 + 2), -4),
    ("rows null", dict(x=None), -5),
    ("q null", dict(q=None), -5),
    ("scales null", dict(s=None), -5),
]


@pytest.mark.parametrize("what,over,code", MX_REJECT, ids=[r[0] for r in MX_REJECT])
def test_mx_rejects(what, over, code):
    a = dict(W=2, M=16, cols=256, dtype=0, x=P16, count=None, q=P16, s=P16)
    a.update(over)
    assert epdc.epdc_mx_quantize(a["W"], a["M"], a["cols"], a["dtype"], a["x"], a["count"], a["q"], a["s"], stream=0,
                                 check=False) == code
    assert epdc.epdc_last_error() != ""
    assert epdc.epdc_mx_dequantize(a["W"], a["M"], a["cols"], a["q"], a["s"], a["count"], a["x"], a["dtype"], stream=0,
                                   check=False) == code


def test_mx_of_nothing():
    assert epdc.epdc_mx_quantize(0, 16, 64, 0, None, None, None, None, stream=0) == 0
    assert epdc.epdc_mx_dequantize(4, 0, 64, None, None, None, None, 0, stream=0) == 0


GROUP_REJECT = [
    ("rank beyond the ranks", {}, 8, {}, -1),
    ("rank -2", {}, -2, {}, -1),
    ("worldSize 65", dict(worldSize=65), 0, {}, -1),
    ("too many slots", dict(maxTokPerRank=1 << 26), 0, {}, -1),
    ("a row of hiddenDim not 16-byte", dict(hiddenDim=7164), 0, {}, -4),
    ("too many experts a rank", dict(numExpertPerRank=1025), 0, {}, -2),
    ("useWeights 2", dict(useWeights=2), 0, {}, -2),
    ("ids misaligned", {}, 0, dict(ids=P16 + 2), -4),
    ("count misaligned", {}, 0, dict(count=P16 + 1), -4),
    ("offsets misaligned", {}, 0, dict(offsets=P16 + 2), -4),
    ("scratch misaligned", {}, 0, dict(scratch=P16 + 4), -4),
    ("ids null", {}, 0, dict(ids=None), -5),
    ("weights null", {}, 0, dict(w=None), -5),
    ("entry weights null", {}, 0, dict(ew=None), -5),
    ("offsets null", {}, 0, dict(offsets=None), -5),
    ("entry rows null", {}, 0, dict(row=None), -5),
    ("entryOf null", {}, 0, dict(of=None), -5),
    ("scratch null", {}, 0, dict(scratch=None), -5),
    ("scratch too small", {}, 0, dict(bytes=64), -6),
]


@pytest.mark.parametrize("what,over,rank,ptrs,code", GROUP_REJECT, ids=[r[0] for r in GROUP_REJECT])
def test_group_rejects(what, over, rank, ptrs, code):
    c = epdc.EpCfg(**{**CFG, **over})
    a = dict(ids=P16, w=P16, count=P16, offsets=P16, row=P16, ew=P16, of=P16, scratch=P16, bytes=1 << 24)
    a.update(ptrs)
    assert epdc.epdc_group_experts(c, rank, a["ids"], a["w"], a["count"], a["offsets"], a["row"], a["ew"], a["of"],
                                   a["scratch"], a["bytes"], stream=0, check=False) == code
    assert epdc.epdc_last_error() != ""


def test_group_scratch_bytes():
    # 4096 rows of 8 slots are 16 tiles of 2048 slots a window; counts per tile and expert, totals per window and expert
    assert epdc.epdc_group_scratch_bytes(epdc.EpCfg(**CFG), 3) == 4 * (8 * 16 * 32 + 8 * 32)
    assert epdc.epdc_group_scratch_bytes(epdc.EpCfg(**{**CFG, "worldSize": 0}), 0) == 0
    assert epdc.epdc_group_scratch_bytes(epdc.EpCfg(**CFG), 8) == 0


PRODUCT_REJECT = [
    ("no experts", dict(E=0), -1),
    ("too many experts", dict(E=65536), -1),
    ("hidden 48", dict(H=48), -1),
    ("hidden beyond the scale limit", dict(H=128 * 1024 + 32), -1),
    ("no columns", dict(N=0), -1),
    ("negative entries", dict(n=-1), -1),
    ("negative rows", dict(R=-1), -1),
    ("bf16 row of 24 bytes", dict(N=12), -4),
    ("fp32 row of 24 bytes", dict(N=6, out_dtype=1), -4),
    ("output fp8", dict(out_dtype=2), -2),
    ("rows misaligned", dict(a=P16 + 8), -4),
    ("weights misaligned", dict(b=P16 + 8), -4),
    ("out misaligned", dict(out=P16 + 8), -4),
    ("row scales misaligned", dict(sa=P16 + 2), -4),
    ("offsets misaligned", dict(offsets=P16 + 2), -4),
    ("entry rows misaligned", dict(row=P16 + 2), -4),
    ("entry weights misaligned", dict(w=P16 + 2), -4),
    ("rows null", dict(a=None), -5),
    ("weight scales null", dict(sb=None), -5),
    ("offsets null", dict(offsets=None), -5),
    ("out null", dict(out=None), -5),
]


@pytest.mark.parametrize("what,over,code", PRODUCT_REJECT, ids=[r[0] for r in PRODUCT_REJECT])
def test_product_rejects(what, over, code):
    v = dict(E=4, N=64, H=256, n=32, R=16, a=P16, sa=P16, offsets=P16, row=P16, w=P16, b=P16, sb=P16, out=P16, out_dtype=0)
    v.update(over)
    assert epdc.epdc_expert_product(v["E"], v["N"], v["H"], v["n"], v["R"], v["a"], v["sa"], v["offsets"], v["row"], v["w"],
                                    v["b"], v["sb"], v["out"], v["out_dtype"], stream=0, check=False) == code
    assert epdc.epdc_last_error() != ""


def test_product_of_nothing():
    assert epdc.epdc_expert_product(4, 64, 256, 0, 0, None, None, None, None, None, None, None, None, 0, stream=0) == 0


def test_host_tensors_are_refused():
    c = epdc.RouteCfg(numExperts=16, numExpertPerToken=2)
    l, ids, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="device"):
        epdc.epdc_route(c, 4, l, None, ids, w, stream=0)
    with pytest.raises(ValueError, match="device"):
        epdc.epdc_mx_quantize(1, 4, 32, epdc.EPDC_FP32, torch.zeros(4, 32), None, P16, P16, stream=0)
