"""What the handles of the grouped products and of the product with adapters refuse, and what they pass on, on the host: real
library checks, tensors that are addresses only, and a recording function in place of the C entry."""
import ctypes

import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod
from test_moe_handles import FakeTensor, fakes  # noqa: F401


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    return B.load()


class Dense(FakeTensor):
    """A dense tensor of any rank."""

    def is_contiguous(self):
        return True


def _recorded(handle, name, problem):
    seen = []

    def entry(ref, *args):
        p = getattr(handle, problem) if isinstance(problem, str) else problem
        seen.append((type(p).from_buffer_copy(p), [a.value for a in args]))
        return 0

    setattr(handle, name, entry)
    return seen


W = (4, 64, 32)  # [E, N, K]


def _grouped(**kw):
    return B.GroupedLinear(Dense(*W), **kw)


def _list(n=4, dtype=torch.int64):
    return Dense(n, dtype=dtype)


def test_the_input_gradient_is_the_product_on_the_weights_the_other_way_round(fakes):  # noqa: F811
    for transposed in (False, True):
        h = _grouped(transposed=transposed)
        N, K = (32, 64) if transposed else (64, 32)
        seen = _recorded(h, "_fn", "_forward")
        y = h(FakeTensor(10, K), _list())
        p, _ = seen[-1]
        assert (p.M, p.N, p.K, p.transposed, p.zero_rest) == (10, N, K, int(transposed), 1) and y.shape == (10, N)
        seen = _recorded(h, "_fn", "_input")
        dx = h.grad_input(FakeTensor(12, N, ld=N + 8), _list())
        p, _ = seen[-1]
        assert (p.M, p.N, p.K, p.ldx, p.transposed) == (12, K, N, N + 8, int(not transposed)) and dx.shape == (12, K)


def test_a_given_output_keeps_its_other_rows(fakes):  # noqa: F811
    h = _grouped()
    seen = _recorded(h, "_fn", "_forward")
    out = FakeTensor(10, 64, ld=72)
    assert h(FakeTensor(10, 32), _list(), out=out) is out
    assert (seen[-1][0].zero_rest, seen[-1][0].ldy) == (0, 72)
    h(FakeTensor(3, 32), _list())
    assert (seen[-1][0].zero_rest, seen[-1][0].ldy, seen[-1][0].M) == (1, 0, 3)


@pytest.mark.parametrize("call", [
    lambda h: h(FakeTensor(10, 64), _list()),  # K is 32
    lambda h: h(FakeTensor(10, 32, dtype=torch.float32), _list()),
    lambda h: h(FakeTensor(10, 32, device=1), _list()),
    lambda h: h(FakeTensor(10, 32, ld=16), _list()),
    lambda h: h(FakeTensor(10, 32), _list(5)),
    lambda h: h(FakeTensor(10, 32), _list(dtype=torch.int32)),
    lambda h: h(FakeTensor(10, 32), _list(), out=FakeTensor(9, 64)),
    lambda h: h(FakeTensor(10, 32), _list(), out=FakeTensor(10, 64, dtype=torch.float32)),
    lambda h: h.grad_input(FakeTensor(10, 32), _list()),  # N is 64
    lambda h: h.grad_weight(FakeTensor(10, 64), FakeTensor(9, 32), _list()),
    lambda h: h.grad_weight(FakeTensor(10, 64), FakeTensor(10, 32), _list(), out=Dense(4, 32, 64)),
    lambda h: h.grad_weight(FakeTensor(10, 64), FakeTensor(10, 32), _list(), out=Dense(*W, dtype=torch.float32)),
    lambda h: h.grad_weight(FakeTensor(10, 64), FakeTensor(10, 32), _list(), accumulate=True)])
def test_grouped_refusals(fakes, call):  # noqa: F811
    with pytest.raises(ValueError):
        call(_grouped())


def test_the_library_refuses_rows_off_boundaries_and_bf16_accumulation(fakes):  # noqa: F811
    h = _grouped()
    for call in (lambda: h(FakeTensor(10, 32, ld=36), _list()), lambda: h(FakeTensor(10, 32, off=8), _list()),
                 lambda: h.grad_weight(FakeTensor(10, 64, ld=68), FakeTensor(10, 32), _list()),
                 lambda: h.grad_weight(FakeTensor(10, 64), FakeTensor(10, 32), _list(), out=Dense(*W), accumulate=True)):
        with pytest.raises(B.GmmfrError) as ei:
            call()
        assert ei.value.status == B.ERR_INVALID_ARG


def test_grouped_weights_and_types(fakes):  # noqa: F811
    for w, kw in ((Dense(4, 64), {}), (Dense(*W, dtype=torch.float32), {}), (Dense(*W), dict(out_dtype=torch.float16)),
                  (Dense(*W), dict(grad_dtype=torch.int32))):
        with pytest.raises(ValueError):
            B.GroupedLinear(w, **kw)
    for w, kw in ((Dense(4, 60, 32), {}), (Dense(1025, 64, 32), {}), (Dense(*W), dict(group_list_type=2))):
        with pytest.raises(B.GmmfrError):
            B.GroupedLinear(w, **kw)


def _lora(rows=64, K=32, count=3, rank=16, **kw):
    return B.LoraLinear(FakeTensor(rows, K), Dense(count, rank, K), Dense(count, rows, rank), **kw)


def test_lora_passes_its_problem_on(fakes):  # noqa: F811
    h = _lora(activation="swiglu", scale=Dense(3, dtype=torch.float32), bias=Dense(64))
    seen = _recorded(h, "_fn", "_p")
    y = h(FakeTensor(10, 32, ld=40), Dense(10, dtype=torch.int32), residual=FakeTensor(10, 32, ld=33))
    p, args = seen[-1]
    q = p.linear
    assert (q.M, q.N, q.K, q.ldx, q.ld_residual, p.count, p.rank) == (10, 32, 32, 40, 33, 3, 16) and y.shape == (10, 32)
    assert len(args) == 12 and all(a for a in args[:10])
    h(FakeTensor(7, 32), Dense(7, dtype=torch.int32))
    p, args = seen[-1]
    assert (p.linear.M, p.linear.ldx, p.linear.ld_residual) == (7, 0, 0) and args[3] is None


@pytest.mark.parametrize("refused", [50, 1000])
def test_lora_runs_the_rows_it_is_given_after_a_refused_call(fakes, refused):  # noqa: F811
    h = _lora()
    seen = _recorded(h, "_fn", "_p")
    h(FakeTensor(100, 32), Dense(100, dtype=torch.int32))
    with pytest.raises(B.GmmfrError):
        h(FakeTensor(refused, 32, ld=36), Dense(refused, dtype=torch.int32))
    h(FakeTensor(100, 32), Dense(100, dtype=torch.int32))
    assert [(p.linear.M, p.linear.ldx) for p, _ in seen] == [(100, 0), (100, 0)]


@pytest.mark.parametrize("call", [
    lambda h: h(FakeTensor(10, 64), Dense(10, dtype=torch.int32)),
    lambda h: h(FakeTensor(10, 32), Dense(9, dtype=torch.int32)),
    lambda h: h(FakeTensor(10, 32), Dense(10, dtype=torch.int64)),
    lambda h: h(FakeTensor(10, 32), Dense(10, dtype=torch.int32, device=1)),
    lambda h: h(FakeTensor(10, 32), Dense(10, dtype=torch.int32), residual=FakeTensor(10, 32)),
    lambda h: h(FakeTensor(10, 32), Dense(10, dtype=torch.int32), out=FakeTensor(10, 64, dtype=torch.float32))])
def test_lora_refusals(fakes, call):  # noqa: F811
    with pytest.raises(ValueError):
        call(_lora())


def test_lora_weights_and_types(fakes):  # noqa: F811
    w, a, b = FakeTensor(64, 32), Dense(3, 16, 32), Dense(3, 64, 16)
    for args, kw in (((w, Dense(3, 16, 40), b), {}), ((w, a, Dense(3, 64, 8)), {}), ((w, a, Dense(2, 64, 16)), {}),
                     ((w, Dense(3, 16), b), {}), ((w, a, b), dict(scale=Dense(2, dtype=torch.float32))),
                     ((w, a, b), dict(scale=Dense(3))), ((w, a, b), dict(bias=Dense(32))), ((w, a, b), dict(activation="tanh")),
                     ((w, a, b), dict(out_dtype=torch.float16)), ((FakeTensor(63, 32), a, Dense(3, 63, 16)), dict(activation="swiglu"))):
        with pytest.raises(ValueError):
            B.LoraLinear(*args, **kw)
    for args in ((w, Dense(3, 12, 32), Dense(3, 64, 12)), (FakeTensor(64, 36), Dense(3, 16, 36), b), (FakeTensor(64, 32, ld=36), a, b)):
        with pytest.raises(B.GmmfrError):
            B.LoraLinear(*args)
    assert ctypes.sizeof(B.LoraProblem) % 8 == 0
