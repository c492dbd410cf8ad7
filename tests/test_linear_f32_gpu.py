"""How exact FP32 results of the dense product are, whatever the length of the sums.

The tensor core's additions truncate: each loses at most 2^-23 of the partial sum, half of that on average, and on average
half of the sum is there.  64 of them (a chunk of 1024 products) take 64 * 2^-24 / 2 = 2^-19 off the chunk's sum, and so off
the total; the chunks are added to nearest (2^-24 each, in either direction).  A gated product has the errors of two
factors, from chunks half as long.  Bound: 2^-19 of the result in the 2-norm.
"""
import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.load()


@pytest.mark.parametrize("K", [40, 264, 1288, 7168, 7175, 30000])
@pytest.mark.parametrize("M,N", [(1, 300), (1, 8192), (7, 5000), (20, 4096), (32, 2048), (48, 300), (64, 2048), (128, 2100), (129, 640),
                                 (300, 2048), (1030, 1500), (2000, 1024)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_long_sums_keep_their_bits(M, N, K, act):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    rows = 2 * N if act == "swiglu" else N
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    w = (torch.randn(rows, K, device="cuda", generator=g) * K ** -0.5).to(torch.bfloat16)
    bias = torch.randn(rows, device="cuda", generator=g).to(torch.bfloat16)
    residual = torch.randn(M, N, device="cuda", generator=g).to(torch.bfloat16)
    y = B.Linear(w, bias=bias, activation=act, out_dtype=torch.float32)(x, residual=residual).double()
    z = x.double() @ w.double().T + bias.double()
    want = (z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:] if act == "swiglu" else z) + residual.double()
    assert (y - want).norm() <= 2.0 ** -19 * want.norm()
