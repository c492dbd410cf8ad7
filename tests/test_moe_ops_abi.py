"""Host-side checks of the router, the few-token layer and the dense product (no GPU): struct sizes and
refusals, each before any CUDA call (the addresses are not real device memory)."""
import ctypes

import pytest

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod

A = 256  # a fake 256-byte-aligned address


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    return B.load()


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(B.GateProblem) == 5 * 8 + 6 * 4 + 4 + 4  # padded to 8
    assert ctypes.sizeof(B.LayerProblem) == ctypes.sizeof(B.GateProblem) + 4 * 8 + 4 + 4
    assert ctypes.sizeof(B.LinearProblem) == 7 * 8 + 3 * 4 + 4


def _gate(**kw):
    base = dict(T=4, H=64, E=32, topk=4, ldx=0, scoring=0, n_group=1, topk_group=1, group_top=2, renormalise=1,
                ids_type=1, scale=1.0)
    base.update(kw)
    return B.GateProblem(**base)


BAD_GATE = [
    (dict(T=-1), "T=-1"), (dict(T=1 << 31), "T="), (dict(H=60), "H=60"), (dict(H=0), "H=0"), (dict(E=0), "E=0"),
    (dict(E=1025), "E=1025"), (dict(topk=0), "topk=0"), (dict(topk=33), "topk=33"), (dict(E=3, topk=4), "topk=4"),
    (dict(ldx=56), "ldx=56"), (dict(ldx=68), "ldx=68"), (dict(scoring=2), "scoring=2"), (dict(n_group=5), "n_group=5"),
    (dict(n_group=0), "n_group=0"), (dict(E=1024, n_group=128), "n_group=128"),
    (dict(n_group=4, topk_group=5), "topk_group=5"), (dict(n_group=4, topk_group=0), "topk_group=0"),
    (dict(n_group=4, group_top=3), "group_top=3"), (dict(n_group=32, topk_group=8, group_top=2), "group_top=2"),
    (dict(n_group=16, topk_group=1), "eligible"), (dict(renormalise=2), "renormalise"), (dict(ids_type=2), "ids_type=2"),
]


@pytest.mark.parametrize("kw,msg", BAD_GATE, ids=[m + str(i) for i, (_, m) in enumerate(BAD_GATE)])
def test_gate_refusals(kw, msg):
    for call in (lambda p: B.gmmfr_moe_gate_workspace_size(p),
                 lambda p: B.gmmfr_moe_gate(p, A, A, None, A, A, None, A, 1 << 40),
                 lambda p: B.gmmfr_moe_layer_workspace_size(B.LayerProblem(gate=p, I=64, weight_type=B.DT_BF16))):
        with pytest.raises(B.GmmfrError) as ei:
            call(_gate(**kw))
        assert ei.value.status == B.ERR_INVALID_ARG and msg in str(ei.value)


def test_gate_pointer_and_workspace_refusals():
    p = _gate()
    need = B.gmmfr_moe_gate_workspace_size(p)
    good = [A, A, None, A, A, None, A, need]
    for i, v, st in ((0, None, B.ERR_INVALID_ARG), (1, None, B.ERR_INVALID_ARG), (3, None, B.ERR_INVALID_ARG),
                     (4, None, B.ERR_INVALID_ARG), (0, A + 8, B.ERR_INVALID_ARG), (1, A + 2, B.ERR_INVALID_ARG),
                     (2, A + 2, B.ERR_INVALID_ARG), (3, A + 2, B.ERR_INVALID_ARG), (6, None, B.ERR_WORKSPACE),
                     (6, A + 128, B.ERR_WORKSPACE), (7, need - 1, B.ERR_WORKSPACE)):
        args = list(good)
        args[i] = v
        with pytest.raises(B.GmmfrError) as ei:
            B.gmmfr_moe_gate(p, *args)
        assert ei.value.status == st
    B.gmmfr_moe_gate(_gate(T=0), None, None, None, None, None, None, None, 0)  # nothing to do


def _layer(gate=None, **kw):
    base = dict(I=64, shared_I=0, ld_residual=0, ld_out=0, weight_type=B.DT_BF16)
    base.update(kw)
    return B.LayerProblem(gate=_gate(**(gate or {})), **base)


@pytest.mark.parametrize("kw,msg", [
    (dict(gate=dict(T=65)), "T=65"), (dict(I=0), "I=0"), (dict(I=60), "I=60"), (dict(shared_I=-8), "I=-8"),
    (dict(shared_I=12), "I=12"), (dict(ld_residual=32), "ld_residual=32"), (dict(ld_out=63), "ld_out=63"),
    (dict(weight_type=B.DT_E5M2), "weight_type"), (dict(weight_type=B.DT_F32), "weight_type")], ids=lambda v: str(v)[:20])
def test_layer_refusals(kw, msg):
    with pytest.raises(B.GmmfrError) as ei:
        B.gmmfr_moe_layer_workspace_size(_layer(**kw))
    assert ei.value.status == B.ERR_INVALID_ARG and msg in str(ei.value)


@pytest.mark.parametrize("wt", [B.DT_BF16, B.DT_E4M3])
def test_layer_pointer_and_buffer_refusals(wt):
    p = _layer(shared_I=128, weight_type=wt)
    need = B.gmmfr_moe_layer_workspace_size(p)
    if wt == B.DT_BF16:
        pb, sb = (B.gmmfr_ffn_prepared_weights_size(B.FfnProblem(N=0, H=64, I=i, E=e)) for i, e in ((64, 32), (128, 1)))
    else:
        pb, sb = (B.gmmfr_ffn_prepared_weights_size_mx(B.FfnProblem(N=0, H=64, I=i, E=e)) for i, e in ((64, 32), (128, 1)))
    good = [A, A, None, None, A, A, pb, A, sb, None, None, A, need]
    bad = [(0, None), (1, None), (4, None), (5, None), (7, None), (0, A + 2), (1, A + 8), (5, A + 8), (7, A + 4), (3, A + 1),
           (4, A + 1), (9, A + 2), (10, A + 2)]
    for i, v in bad:
        args = list(good)
        args[i] = v
        with pytest.raises(B.GmmfrError) as ei:
            B.gmmfr_moe_layer(p, *args)
        assert ei.value.status == B.ERR_INVALID_ARG, (i, v)
    for i, v in ((6, pb - 1), (8, sb - 1), (11, None), (11, A + 16), (12, need - 1)):
        args = list(good)
        args[i] = v
        with pytest.raises(B.GmmfrError) as ei:
            B.gmmfr_moe_layer(p, *args)
        assert ei.value.status == B.ERR_WORKSPACE, (i, v)
    B.gmmfr_moe_layer(_layer(gate=dict(T=0)), None, None, None, None, None, None, 0, None, 0, None, None, None, 0)


def test_mx_weight_preparation_refusals():
    p = B.FfnProblem(N=0, H=64, I=64, E=2)
    n = B.gmmfr_ffn_prepared_weights_size_mx(p)
    assert n == 2 * (1 * 1 + 1 * 1) * 16896
    for args, st in (((None, A, A, A, A, n), B.ERR_INVALID_ARG), ((A, A, A, A, None, n), B.ERR_INVALID_ARG),
                     ((A, A, A, A, A, n - 1), B.ERR_WORKSPACE), ((A, A, A, A, A + 8, n), B.ERR_WORKSPACE)):
        with pytest.raises(B.GmmfrError) as ei:
            B.gmmfr_ffn_prepare_weights_mx(p, *args)
        assert ei.value.status == st
    with pytest.raises(B.GmmfrError):
        B.gmmfr_ffn_prepared_weights_size_mx(B.FfnProblem(N=0, H=62, I=64, E=2))


def _linear(**kw):
    base = dict(M=4, N=16, K=32, ldx=0, ldw=0, ld_residual=0, ld_out=0, activation=0, out_type=B.DT_BF16)
    base.update(kw)
    return B.LinearProblem(**base)


@pytest.mark.parametrize("kw,msg", [
    (dict(M=-1), "M=-1"), (dict(N=-1), "N=-1"), (dict(K=0), "K=0"), (dict(M=1 << 31), "M="), (dict(N=1 << 30), "N="),
    (dict(ldx=31), "ldx=31"), (dict(ldw=8), "ldw=8"), (dict(ld_residual=15), "ld_residual=15"), (dict(ld_out=1), "ld_out=1"),
    (dict(activation=6), "activation=6"), (dict(activation=-1), "activation"), (dict(unaligned=2), "unaligned"), (dict(out_type=B.DT_U8), "out_type")],
    ids=lambda v: str(v)[:24])
def test_linear_refusals(kw, msg):
    for call in (lambda p: B.gmmfr_linear_workspace_size(p), lambda p: B.gmmfr_linear(p, A, A, None, None, A, A, 1 << 40)):
        with pytest.raises(B.GmmfrError) as ei:
            call(_linear(**kw))
        assert ei.value.status == B.ERR_INVALID_ARG and msg in str(ei.value)


def test_linear_pointer_refusals():
    for args in ((None, A, None, None, A), (A, None, None, None, A), (A, A, None, None, None), (A + 1, A, None, None, A),
                 (A, A + 1, None, None, A), (A, A, A + 1, None, A), (A, A, None, A + 1, A), (A, A, None, None, A + 1)):
        with pytest.raises(B.GmmfrError) as ei:
            B.gmmfr_linear(_linear(), *args, A, 1 << 40)
        assert ei.value.status == B.ERR_INVALID_ARG
    with pytest.raises(B.GmmfrError):  # a float32 out on a 2-byte boundary
        B.gmmfr_linear(_linear(out_type=B.DT_F32), A, A, None, None, A + 2, A, 1 << 40)
    for args, msg in (((A + 2, A, None, None, A), "unaligned"), ((A, A + 8, None, None, A), "unaligned")):
        with pytest.raises(B.GmmfrError, match=msg):
            B.gmmfr_linear(_linear(), *args, A, 1 << 40)
    big = B.gmmfr_linear_workspace_size(_linear(unaligned=1))
    assert big > B.gmmfr_linear_workspace_size(_linear()) == 4096
    for p, ws, n in ((_linear(), None, 1 << 20), (_linear(), A + 8, 1 << 20), (_linear(), A, 4095), (_linear(unaligned=1), A, big - 1),
                     (_linear(K=33), A, 4096)):
        with pytest.raises(B.GmmfrError) as ei:
            B.gmmfr_linear(p, A, A, None, None, A, ws, n)
        assert ei.value.status == B.ERR_WORKSPACE
    B.gmmfr_linear(_linear(M=0), None, None, None, None, None, None, 0)
    B.gmmfr_linear(_linear(N=0), None, None, None, None, None, None, 0)
