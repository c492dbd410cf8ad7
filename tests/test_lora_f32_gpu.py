"""FP32 results of the product with adapters keep their bits where the adapters' ranks are many: what an adapter adds is a sum of its
own, not a tail of the last of the dense product's.

All terms are of one sign, so that truncation adds up: n additions of 16 products by the tensor core take at most
2^-23 * (1 + ... + n) / n = (n + 1) / 2 * 2^-23 off their sum.  The dense product's sums are of at most 1024 products, and so are
those of x A^T; the adapter's are rank / 16 additions of each of the three BF16 numbers that a sum x A^T is.  (One such addition of
each, up to rank 16, may be onto the dense product's last sum: 3 * 2^-23 of it.)  All of these are added to nearest, a few times 2^-24
(taken as 2^-22).  SwiGLU of large positive numbers is their product: both errors, and 2^-20 of its value
for the exponential and division.
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


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("K,r", [(256, 256), (1024, 256), (1024, 64), (4096, 256), (4096, 8)])
@pytest.mark.parametrize("M,N", [(20, 320), (100, 320), (128, 4096), (300, 512), (1030, 4096)])
def test_ranks_have_sums_of_their_own(M, N, K, r, act):
    g = torch.Generator(device="cuda").manual_seed(M + K + r)
    rows = 2 * N if act == "swiglu" else N
    x = torch.randn(M, K, device="cuda", generator=g).abs().to(torch.bfloat16)
    w = torch.rand(rows, K, device="cuda", generator=g).to(torch.bfloat16)
    a = (torch.rand(3, r, K, device="cuda", generator=g) / K).to(torch.bfloat16)
    b = torch.rand(3, rows, r, device="cuda", generator=g).to(torch.bfloat16)
    ids = (torch.arange(M, device="cuda") % 4 - 1).to(torch.int32)
    y = B.LoraLinear(w, a, b, activation=act, out_dtype=torch.float32)(x, ids).double()
    dense = x.double() @ w.double().T
    more = torch.zeros_like(dense)
    for i in range(3):
        more[ids == i] = (x[ids == i].double() @ a[i].double().T) @ b[i].double().T

    def lost(n):
        return (n + 1) / 2 * 2.0 ** -23

    long = lost(min(K, 1024) / 16) + (3 * 2.0 ** -23 if r <= 16 else 0)
    z, off = dense + more, long * dense + (long + lost(3 * r / 16)) * more + 2.0 ** -22 * (dense + more)
    if act == "swiglu":
        gate, up = z[:, :N], z[:, N:]
        off = off[:, :N] * up + off[:, N:] * gate + 2.0 ** -20 * gate * up
        z = gate * torch.sigmoid(gate) * up
    assert ((y - z).abs() <= off).all(), float(((y - z).abs() / off).max())
