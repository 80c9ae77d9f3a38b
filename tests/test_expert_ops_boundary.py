"""Host checks of the experts in bf16 and int8: every refusal with its
documented code before anything is launched, and the binding's own checks of
its tensors.  No GPU is needed."""
import os
import re

import pytest
import torch

import combine_count_amd as epdc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P16 = 0x10000  # a fake, 16-byte aligned device address: never dereferenced on these paths


def test_header_constant():
    src = open(os.path.join(ROOT, "include", "epdc.h")).read()
    assert int(re.search(r"EPDC_MAX_EXPERT_DIM (\d+)", src).group(1)) == epdc.EPDC_MAX_EXPERT_DIM


PRODUCT = dict(E=4, N=64, H=256, n=32, R=16, x=P16, sx=P16, offsets=P16, row=P16, w=P16, b=P16, sb=P16, out=P16, dtype=0)
SHARED = [
    ("no experts", dict(E=0), -1),
    ("too many experts", dict(E=65536), -1),
    ("no hidden", dict(H=0), -1),
    ("hidden beyond the limit", dict(H=131072), -1),
    ("no columns", dict(N=0), -1),
    ("too many columns", dict(N=(1 << 20) + 16), -1),
    ("negative entries", dict(n=-1), -1),
    ("entries beyond the limit", dict(n=2 ** 31 - 1), -1),
    ("negative rows", dict(R=-1), -1),
    ("hidden 100", dict(H=100), -4),
    ("columns 12 in bf16", dict(N=12), -4),
    ("columns 6 in fp32", dict(N=6, dtype=1), -4),
    ("output fp8", dict(dtype=2), -2),
    ("output 7", dict(dtype=7), -2),
    ("rows misaligned", dict(x=P16 + 8), -4),
    ("weights misaligned", dict(b=P16 + 8), -4),
    ("out misaligned", dict(out=P16 + 8), -4),
    ("offsets misaligned", dict(offsets=P16 + 2), -4),
    ("entry rows misaligned", dict(row=P16 + 1), -4),
    ("entry weights misaligned", dict(w=P16 + 2), -4),
    ("rows null", dict(x=None), -5),
    ("weights null", dict(b=None), -5),
    ("offsets null", dict(offsets=None), -5),
    ("out null", dict(out=None), -5),
]
INT8 = [
    ("hidden 24 in int8", dict(H=24), -4),
    ("row scales null", dict(sx=None), -5),
    ("weight scales null", dict(sb=None), -5),
    ("row scales misaligned", dict(sx=P16 + 2), -4),
    ("weight scales misaligned", dict(sb=P16 + 1), -4),
]


def _product(v):
    return epdc.epdc_expert_linear(v["E"], v["N"], v["H"], v["n"], v["R"], v["x"], v["offsets"], v["row"], v["w"], v["b"],
                                         v["out"], v["dtype"], stream=0, check=False)


def _rows_grad(v):
    return epdc.epdc_expert_rows_grad(v["E"], v["N"], v["H"], v["n"], v["R"], v["x"], v["offsets"], v["row"], v["w"], v["b"],
                                      v["out"], v["dtype"], stream=0, check=False)


def _int8(v):
    return epdc.epdc_expert_linear_int(v["E"], v["N"], v["H"], v["n"], v["R"], v["x"], v["sx"], v["offsets"], v["row"], v["w"],
                                         v["b"], v["sb"], v["out"], v["dtype"], stream=0, check=False)


@pytest.mark.parametrize("what,over,code", SHARED, ids=[r[0] for r in SHARED])
@pytest.mark.parametrize("call", [_product, _rows_grad, _int8])
def test_products_reject(call, what, over, code):
    assert call({**PRODUCT, **over}) == code
    assert epdc.epdc_last_error() != ""


@pytest.mark.parametrize("what,over,code", INT8, ids=[r[0] for r in INT8])
def test_int8_product_rejects(what, over, code):
    assert _int8({**PRODUCT, **over}) == code
    assert epdc.epdc_last_error() != ""


def test_rows_grad_takes_columns_by_eight():
    assert _rows_grad({**PRODUCT, "N": 12, "dtype": 1}) == -4  # a row of dOut is not a multiple of 16 bytes


def test_products_of_nothing():
    none = dict(PRODUCT, n=0, x=None, offsets=None, b=None, out=None, sx=None, sb=None, row=None, w=None)
    for call in (_product, _rows_grad, _int8):
        assert call(none) == 0


GRAD = dict(E=4, N=64, H=256, n=32, D=16, d=P16, drow=P16, R=16, x=P16, row=P16, offsets=P16, base=P16, out=P16, dtype=0)


def _weights_grad(v):
    return epdc.epdc_expert_weights_grad(v["E"], v["N"], v["H"], v["n"], v["D"], v["d"], v["drow"], v["R"], v["x"], v["row"],
                                         v["offsets"], v["base"], v["out"], v["dtype"], stream=0, check=False)


@pytest.mark.parametrize("what,over,code", [
    ("no experts", dict(E=0), -1), ("too many experts", dict(E=65536), -1), ("no hidden", dict(H=0), -1),
    ("hidden beyond the limit", dict(H=131072), -1), ("no columns", dict(N=0), -1), ("negative entries", dict(n=-1), -1),
    ("negative rows", dict(R=-1), -1), ("negative output rows", dict(D=-1), -1), ("hidden 100", dict(H=100), -4),
    ("columns 12", dict(N=12, dtype=1), -4), ("fp4 output", dict(dtype=3), -2), ("dOut misaligned", dict(d=P16 + 8), -4),
    ("rows misaligned", dict(x=P16 + 4), -4), ("base misaligned", dict(base=P16 + 8), -4), ("out misaligned", dict(out=P16 + 2), -4),
    ("offsets misaligned", dict(offsets=P16 + 2), -4), ("output rows misaligned", dict(drow=P16 + 2), -4),
    ("entry rows misaligned", dict(row=P16 + 2), -4), ("dOut null", dict(d=None), -5), ("rows null", dict(x=None), -5),
    ("offsets null", dict(offsets=None), -5), ("out null", dict(out=None), -5),
])
def test_weights_grad_rejects(what, over, code):
    assert _weights_grad({**GRAD, **over}) == code
    assert epdc.epdc_last_error() != ""


GATE = dict(E=4, F=64, n=32, dtype=0, h=P16, offsets=P16, w=P16, d=P16, out=P16, out_dtype=0, per=P16)


def _gate(v):
    return epdc.epdc_expert_gate(v["E"], v["F"], v["n"], v["dtype"], v["h"], v["offsets"], v["w"], v["out"], v["out_dtype"],
                                 stream=0, check=False)


def _gate_grad(v):
    return epdc.epdc_expert_gate_grad(v["E"], v["F"], v["n"], v["dtype"], v["h"], v["offsets"], v["w"], v["d"], v["out_dtype"],
                                      v["out"], v["per"], stream=0, check=False)


def _gate_int8(v):
    return epdc.epdc_expert_gate_int(v["E"], v["F"], v["n"], v["dtype"], v["h"], v["offsets"], v["w"], v["out"], v["per"],
                                      stream=0, check=False)


@pytest.mark.parametrize("what,over,code", [
    ("no experts", dict(E=0), -1), ("no columns", dict(F=0), -1), ("too many columns", dict(F=131072), -1),
    ("negative entries", dict(n=-1), -1), ("entries beyond the limit", dict(n=2 ** 31 - 65535), -1),
    ("columns 12", dict(F=12), -4), ("fp8", dict(dtype=2), -2), ("type -1", dict(dtype=-1), -2),
    ("h misaligned", dict(h=P16 + 8), -4), ("out misaligned", dict(out=P16 + 8), -4), ("offsets misaligned", dict(offsets=P16 + 2), -4),
    ("weights misaligned", dict(w=P16 + 2), -4), ("h null", dict(h=None), -5), ("out null", dict(out=None), -5),
])
@pytest.mark.parametrize("call", [_gate, _gate_grad, _gate_int8])
def test_gates_reject(call, what, over, code):
    assert call({**GATE, **over}) == code
    assert epdc.epdc_last_error() != ""


def test_gates_reject_their_own():
    assert _gate({**GATE, "out_dtype": 2}) == -2 and _gate_grad({**GATE, "out_dtype": 4}) == -2
    assert _gate_grad({**GATE, "d": None}) == -5 and _gate_grad({**GATE, "d": P16 + 8}) == -4
    assert _gate_grad({**GATE, "per": P16 + 2}) == -4 and _gate_int8({**GATE, "per": P16 + 2}) == -4
    assert _gate_int8({**GATE, "per": None}) == -5
    assert _gate_int8({**GATE, "F": 24}) == -4
    for call in (_gate, _gate_grad, _gate_int8):
        assert call(dict(GATE, n=0, h=None, out=None, d=None, per=None)) == 0


@pytest.mark.parametrize("what,over,code", [
    ("negative windows", dict(W=-1), -1), ("negative rows", dict(M=-1), -1), ("too many rows", dict(W=1 << 16, M=1 << 15), -1),
    ("cols 0", dict(cols=0), -1), ("cols beyond the limit", dict(cols=131072), -1), ("cols 24", dict(cols=24), -4),
    ("fp4x2", dict(dtype=3), -2), ("x misaligned", dict(x=P16 + 8), -4), ("q misaligned", dict(q=P16 + 4), -4),
    ("scales misaligned", dict(s=P16 + 2), -4), ("count misaligned", dict(count=P16 + 2), -4), ("x null", dict(x=None), -5),
    ("q null", dict(q=None), -5), ("scales null", dict(s=None), -5),
])
def test_int_quantize_rejects(what, over, code):
    v = dict(W=2, M=16, cols=256, dtype=0, x=P16, count=None, q=P16, s=P16)
    v.update(over)
    assert epdc.epdc_int_quantize(v["W"], v["M"], v["cols"], v["dtype"], v["x"], v["count"], v["q"], v["s"], stream=0,
                                   check=False) == code
    assert epdc.epdc_last_error() != ""
    assert epdc.epdc_int_quantize(0, 16, 64, 0, None, None, None, None, stream=0) == 0


def test_host_tensors_and_wide_integers_are_refused():
    t = torch.zeros(64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        epdc.epdc_expert_gate(1, 32, 64, epdc.EPDC_BF16, t, None, None, P16, epdc.EPDC_BF16, stream=0)
    with pytest.raises(ValueError, match="device"):
        epdc.epdc_expert_linear(1, 64, 64, 64, 64, t, P16, None, None, P16, P16, epdc.EPDC_BF16, stream=0)
    with pytest.raises(ValueError, match="32 bits"):
        epdc.epdc_expert_gate(1, 32, 1 << 31, epdc.EPDC_BF16, P16, None, None, P16, epdc.EPDC_BF16, stream=0)


def test_the_largest_number_of_entries():
    src = open(os.path.join(ROOT, "include", "epdc.h")).read()
    limit = epdc.EPDC_MAX_EXPERT_ENTRIES
    assert int(re.search(r"EPDC_MAX_EXPERT_ENTRIES (\d+)", src).group(1)) == limit
    assert "EPDC_MAX_EXPERT_ENTRIES" in epdc.__all__
    for call in (_product, _rows_grad, _int8):  # the limit itself passes this check and meets the next
        assert call({**PRODUCT, "n": limit + 1}) == -1 and call({**PRODUCT, "n": limit, "x": None}) == -5
    for call in (_gate, _gate_grad, _gate_int8):
        assert call({**GATE, "n": limit + 1}) == -1 and call({**GATE, "n": limit, "h": None}) == -5
    assert _weights_grad({**GRAD, "n": limit + 1}) == -1 and _weights_grad({**GRAD, "n": limit, "d": None}) == -5
