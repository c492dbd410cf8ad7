"""Host-side checks of the products grouped by expert (no GPU): struct size and refusals, each before any CUDA call (the
addresses are not real device memory)."""
import ctypes

import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod

A = 256  # a fake 256-byte-aligned address


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    return B.load()


def _problem(**kw):
    base = dict(M=64, N=128, K=64, E=4, group_list_type=1, out_type=B.DT_BF16)
    base.update(kw)
    return B.GroupedProblem(**base)


def _product(p, x=A, w=A, g=A, y=A, ws=A, n=4096):
    B.gmmfr_grouped_linear(p, x, w, g, y, ws, n)


def _grad(p, dy=A, x=A, g=A, dw=A, ws=A, n=1 << 20):
    B.gmmfr_grouped_linear_grad_weight(p, dy, x, g, dw, ws, n)


def test_struct_size_matches_the_header():
    assert ctypes.sizeof(B.GroupedProblem) == 6 * 8 + 5 * 4 + 4  # padded to 8


BAD = [
    (dict(M=-1), "M=-1"), (dict(M=1 << 31), "M="), (dict(N=0), "N=0"), (dict(N=12), "N=12"), (dict(K=4), "K=4"), (dict(K=-8), "K=-8"),
    (dict(N=1 << 24), "N="), (dict(N=(1 << 24) - 8, K=1 << 15), "2^38"), (dict(E=0), "E=0"), (dict(E=1025), "E=1025"),
    (dict(ldx=56), "ldx=56"), (dict(ldx=68), "ldx=68"), (dict(ldy=120), "ldy=120"), (dict(ldx=1 << 38), "2^38"),
    (dict(transposed=2), "transposed"), (dict(group_list_type=2), "group_list_type"), (dict(out_type=B.DT_E4M3), "out_type"),
    (dict(zero_rest=2), "zero_rest"), (dict(accumulate=-1), "accumulate"),
]


def test_row_numbers_stay_within_32_bits():
    assert B.gmmfr_grouped_linear_workspace_size(_problem(M=(1 << 31) - 1024)) > 0
    for call in (B.gmmfr_grouped_linear_workspace_size, _product, _grad):
        with pytest.raises(B.GmmfrError, match="M=2147482625"):
            call(_problem(M=(1 << 31) - 1023))


@pytest.mark.parametrize("kw,msg", BAD, ids=[m + str(i) for i, (_, m) in enumerate(BAD)])
def test_refused_problems(kw, msg):
    for call in (B.gmmfr_grouped_linear_workspace_size, _product, _grad):
        with pytest.raises(B.GmmfrError) as ei:
            call(_problem(**kw))
        assert ei.value.status == B.ERR_INVALID_ARG and msg in str(ei.value)


@pytest.mark.parametrize("kw,msg", [
    (dict(x=None), "non-NULL"), (dict(w=None), "non-NULL"), (dict(g=None), "non-NULL"), (dict(y=None), "non-NULL"),
    (dict(x=A + 8), "16-byte"), (dict(w=A + 2), "16-byte"), (dict(g=A + 4), "element size"), (dict(y=A + 1), "element size"),
    (dict(ws=None), "workspace"), (dict(ws=A + 16), "256-byte"), (dict(n=4095), "4095")], ids=lambda v: str(v)[:24])
def test_refused_arguments_of_the_product(kw, msg):
    with pytest.raises(B.GmmfrError) as ei:
        _product(_problem(), **kw)
    assert msg in str(ei.value) and ei.value.status == (B.ERR_WORKSPACE if "ws" in kw or "n" in kw else B.ERR_INVALID_ARG)


@pytest.mark.parametrize("kw,msg", [
    (dict(x=None), "non-NULL"), (dict(dy=None), "non-NULL"), (dict(g=None), "non-NULL"), (dict(dw=None), "dweight"),
    (dict(x=A + 8), "16-byte"), (dict(dy=A + 2), "16-byte"), (dict(dw=A + 8), "16-byte"), (dict(g=A + 4), "element size"),
    (dict(ws=None), "workspace"), (dict(ws=A + 16), "256-byte"), (dict(n=4095), "4095")], ids=lambda v: str(v)[:24])
def test_refused_arguments_of_the_gradient(kw, msg):
    with pytest.raises(B.GmmfrError) as ei:
        _grad(_problem(), **kw)
    assert msg in str(ei.value) and ei.value.status == (B.ERR_WORKSPACE if "ws" in kw or "n" in kw else B.ERR_INVALID_ARG)


def test_options_of_the_other_call_are_refused():
    for call, kw, msg in ((_product, dict(accumulate=1, out_type=B.DT_F32), "accumulate"), (_grad, dict(zero_rest=1), "zero_rest"),
                          (_grad, dict(accumulate=1), "FP32"), (_grad, dict(ldy=132), "ldy=132")):
        with pytest.raises(B.GmmfrError) as ei:
            call(_problem(**kw))
        assert ei.value.status == B.ERR_INVALID_ARG and msg in str(ei.value)


def test_nothing_to_do():
    _product(_problem(M=0), None, None, None, None, None, 0)
    _grad(_problem(M=0, accumulate=1, out_type=B.DT_F32), None, None, None, None, None, 0)


def test_the_handle_refuses_what_it_does_not_take():
    w = torch.zeros(2, 16, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.GroupedLinear(w)  # not on a device
