"""Integer arguments beyond 32 bits are refused, not cut to their low half.
No GPU is needed: nothing is launched."""
import pytest

import combine_count_amd as epdc

P16 = 0x10000  # a fake, 16-byte aligned device address: never dereferenced on these paths
C = epdc.RouteCfg(numExperts=16, numExpertPerToken=2)
D = epdc.EpCfg(worldSize=2, hiddenDim=64, maxTokPerRank=8, numExpertPerRank=2, numExpertPerToken=2, dtype=0, useWeights=0,
               scaleDim=0)
BIG = 2 ** 32  # 0 in its low 32 bits: a call of nothing, or rank 0


@pytest.mark.parametrize("call", [
    lambda: epdc.epdc_route(C, BIG, P16, None, P16, P16, stream=0),
    lambda: epdc.epdc_route_grad(C, -BIG, P16, P16, P16, P16, stream=0),
    lambda: epdc.epdc_mx_quantize(BIG, 16, 64, 0, P16, None, P16, P16, stream=0),
    lambda: epdc.epdc_mx_quantize(1, BIG, 64, 0, P16, None, P16, P16, stream=0),
    lambda: epdc.epdc_mx_dequantize(1, 0, BIG + 64, P16, P16, None, P16, 0, stream=0),
    lambda: epdc.epdc_group_scratch_bytes(D, BIG),
    lambda: epdc.epdc_group_experts(D, BIG, P16, None, P16, P16, P16, None, P16, P16, 0, stream=0),
    lambda: epdc.epdc_expert_product(2, 64, 64, BIG, 8, P16, P16, P16, P16, P16, P16, P16, P16, 0, stream=0),
])
def test_integers_beyond_32_bits(call):
    with pytest.raises(ValueError, match="32 bits"):
        call()


def test_scale_dim_beyond_32_bits():
    assert [epdc.epdc_mx_scale_dim(c) for c in (BIG + 32, -BIG + 32, 2 ** 31 + 32)] == [-1] * 3
