"""Host-side checks of the dense product with adapters (no GPU): struct size and refusals, each before any CUDA call (the
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


def _problem(count=4, rank=16, **kw):
    base = dict(M=8, N=64, K=64, activation=B.ACTIVATIONS["none"], out_type=B.DT_BF16)
    base.update(kw)
    return B.LoraProblem(linear=B.LinearProblem(**base), count=count, rank=rank)


def _call(p, x=A, w=A, bias=None, res=None, a=A, b=A, scale=A, ids=A, out=A, ws=A, n=1 << 30):
    B.gmmfr_lora_linear(p, x, w, bias, res, a, b, scale, ids, out, ws, n)


def test_struct_size_matches_the_header():
    assert ctypes.sizeof(B.LoraProblem) == ctypes.sizeof(B.LinearProblem) + 2 * 8


@pytest.mark.parametrize("kw,msg", [
    (dict(M=-1), "M=-1"), (dict(K=60), "K=60"), (dict(ldx=68), "ldx=68"), (dict(ldw=71), "ldw=71"), (dict(ldx=56), "ldx=56"),
    (dict(unaligned=1), "unaligned"), (dict(activation=9), "activation=9"), (dict(out_type=B.DT_U8), "out_type"),
    (dict(count=0), "count=0"), (dict(count=1 << 24), "count="), (dict(rank=0), "rank=0"), (dict(rank=12), "rank=12"),
    (dict(rank=264), "rank=264"), (dict(rank=-8), "rank=-8")], ids=lambda v: str(v)[:20])
def test_refused_problems(kw, msg):
    for call in (B.gmmfr_lora_linear_workspace_size, _call):
        with pytest.raises(B.GmmfrError) as ei:
            call(_problem(**kw))
        assert ei.value.status == B.ERR_INVALID_ARG and msg in str(ei.value)


@pytest.mark.parametrize("kw,msg", [
    (dict(x=None), "non-NULL"), (dict(w=None), "non-NULL"), (dict(out=None), "non-NULL"), (dict(a=None), "non-NULL"),
    (dict(b=None), "non-NULL"), (dict(ids=None), "non-NULL"), (dict(x=A + 8), "16-byte"), (dict(w=A + 8), "16-byte"),
    (dict(a=A + 8), "16-byte"), (dict(b=A + 8), "16-byte"), (dict(scale=A + 2), "element size"), (dict(ids=A + 2), "element size"),
    (dict(bias=A + 1), "element size"), (dict(res=A + 1), "element size"), (dict(out=A + 1), "element size")],
    ids=lambda v: str(v)[:20])
def test_refused_arguments(kw, msg):
    with pytest.raises(B.GmmfrError) as ei:
        _call(_problem(), **kw)
    assert ei.value.status == B.ERR_INVALID_ARG and msg in str(ei.value)


def test_refused_workspaces():
    need = B.gmmfr_lora_linear_workspace_size(_problem())
    assert need >= 4096 + 8 * 16 * 4
    for kw in (dict(ws=None), dict(ws=A + 128), dict(n=need - 1)):
        with pytest.raises(B.GmmfrError) as ei:
            _call(_problem(), **kw)
        assert ei.value.status == B.ERR_WORKSPACE


def test_nothing_to_do():
    _call(_problem(M=0), None, None, None, None, None, None, None, None, None, None, 0)
    _call(_problem(N=0), None, None, None, None, None, None, None, None, None, None, 0)


def test_the_handle_refuses_what_it_does_not_take():
    w, a, b = (torch.zeros(s, dtype=torch.bfloat16) for s in ((16, 8), (2, 8, 8), (2, 16, 8)))
    with pytest.raises(ValueError):
        B.LoraLinear(w, a, b)  # not on a device
