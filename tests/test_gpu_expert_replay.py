"""A captured step of a sparse layer follows its inputs: replayed with other
tokens, other routing (other groups, counts and weights) and other gradients,
with eager steps of another layer and synchronisations in between, every replay
gives what an eager step gives on the same inputs."""
import pytest
import torch

from test_gpu_expert_layer import Layer

pytestmark = pytest.mark.gpu

INPUTS = ("x", "logits", "dy")
POISONED = ("h1", "a", "y2", "yrow", "y", "da", "dh1", "dwgt", "dx2", "dxrow", "dx", "dw1", "dw2")


def _set(layer, inputs):
    for name, value in inputs.items():
        getattr(layer, name).copy_(value)


def test_replays_follow_changed_inputs():
    layer, other = Layer(11), Layer(12)
    first = {k: getattr(layer, k).clone() for k in INPUTS}
    inputs = [first, {**first, "logits": -first["logits"]}, {k: getattr(other, k).clone() for k in INPUTS},
              {"x": first["x"].flip(0), "logits": first["logits"].roll(3, 1), "dy": -first["dy"]}]
    wants = []
    for given in inputs:
        _set(layer, given)
        layer.run()
        torch.cuda.synchronize()
        wants.append({k: v.clone() for k, v in layer.results().items()})
    assert len({tuple(w["ids"].flatten().tolist()) for w in wants}) == len(inputs)  # other groups each time
    assert len({tuple(w["dw1"].flatten()[:50].tolist()) for w in wants}) == len(inputs)
    _set(layer, inputs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run()
    for i, at in enumerate((1, 2, 0, 3, 1, 1, 2, 0)):
        _set(layer, inputs[at])
        for name in POISONED:
            getattr(layer, name).fill_(float("nan") if i % 2 else 3.0)
        if i % 3 == 1:
            other.run()
            torch.cuda.synchronize()
        graph.replay()
        if i % 3 != 2:
            torch.cuda.synchronize()
        for k, v in layer.results().items():
            assert torch.equal(v, wants[at][k]), (i, at, k)
