"""What a prepared call keeps: its configuration as it was checked, whatever
becomes of the caller's object.  No GPU is needed: calls without tokens
launch nothing, and a refusal launches nothing."""
import pytest

import combine_count_amd as epdc

P16 = 0x10000  # a fake, 16-byte aligned device address: never dereferenced on these paths


def _dispatch_cfg():
    return epdc.EpCfg(worldSize=2, hiddenDim=64, maxTokPerRank=8, numExpertPerRank=2, numExpertPerToken=2, dtype=0, useWeights=0,
                      scaleDim=0)


ROUTE = dict(numExperts=16, numExpertPerToken=2)
CALLS = {
    # (make the configuration, prepare, what it returns, the field that a later change breaks)
    "route": (lambda: epdc.RouteCfg(**ROUTE), lambda c: epdc.prepare_route(c, 0, None, None, None, None), 0, "numExperts"),
    "route_grad": (lambda: epdc.RouteCfg(**ROUTE), lambda c: epdc.prepare_route_grad(c, 0, None, None, None, None), 0, "numExperts"),
    "combine": (_dispatch_cfg, lambda c: epdc.prepare_combine(c, 0, None, None, None, None, None), 0, "worldSize"),
    "combine_push": (_dispatch_cfg, lambda c: epdc.prepare_combine_push(c, 0, None, None, None, None, None, None), 0, "worldSize"),
    "combine_reduce": (_dispatch_cfg, lambda c: epdc.prepare_combine_reduce(c, 0, None, None, None, None, None), 0, "worldSize"),
    # refused for their scratch, behind the checks of the configuration
    "dispatch": (_dispatch_cfg, lambda c: epdc.prepare_dispatch(c, 8, *[P16] * 2, None, None, P16, P16, P16, None, None, P16, P16, P16,
                                                                scratchBytes=0), -6, "worldSize"),
    "group": (_dispatch_cfg, lambda c: epdc.prepare_group_experts(c, 0, P16, None, P16, P16, P16, None, P16, P16, 0), -6, "worldSize"),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_prepared_call_keeps_its_configuration(name):
    make, prepare, code, field = CALLS[name]
    cfg = make()
    call = prepare(cfg)
    assert call(stream=0, check=False) == code
    setattr(cfg, field, 0)
    assert prepare(cfg)(stream=0, check=False) == -1  # the change is one that is refused
    assert call(stream=0, check=False) == code
