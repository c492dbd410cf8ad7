"""The example block: its two ways through the operators, each against the float64 oracle.

Tolerance: the SwiGLU value, each expert's result and the shared expert's are rounded to BF16 (2^-9 of a term each, with
what the sums leave 2^-7 of their absolute sum), the result and the residual's sum once more (2^-8).
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod
from oracle import moe as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.load()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


@pytest.mark.parametrize("T", [1, 9, 64, 150])
def test_block(example, T):
    weights, block = example.random_block(E=16, H=256, I=128, shared_I=192, topk=3, seed=T)
    g = torch.Generator().manual_seed(T)
    x, residual = (torch.randn(T, 256, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    ids, wt = block.gate(x)
    w = {k: _f64(v) for k, v in weights.items()}
    ref, absb = O.moe_layer(_f64(x), ids.cpu().numpy(), _f64(wt), w["w13"], w["w2"], w["shared_w13"], w["shared_w2"],
                            residual=_f64(residual))
    tol = 2.0 ** -7 * absb + 2.0 ** -8 * (np.abs(ref) + np.abs(_f64(residual)))
    assert np.all(np.abs(_f64(block.prefill(x, residual)) - ref) <= tol)
    if T <= 64:
        assert np.all(np.abs(_f64(block.decode(x, residual)) - ref) <= tol)
