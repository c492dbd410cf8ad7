"""How exact the sums x A^T of the product with adapters are for FP32 results, whatever their length and however the rows are shared
out: as the dense product's.

The base weight is zero and the second factor copies a row's sums to the outputs (y[n] = s[n % rank], exact: a sum enters the product
as three BF16 numbers that leave nothing out, whose two additions may truncate by 2^-23 each).  x and A are of one sign, so that
truncation adds up: 1024 products are 64 additions of 16 by the tensor core, each at most 2^-23 off a running sum that is i / 64 of
the whole: (1 + ... + 64) / 64 * 2^-23 = 32.5 * 2^-23 of it.  Longer sums are of such sums, added to nearest, 2^-25 each in either
direction: 200 of them come to 2^-21 in the 2-norm.  In one accumulator 7168 products could lose 224.5 * 2^-23.
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


def _sums(M, K, L, N=64, rank=8, scale=None):
    """The sums as they come out in FP32 (rows of adapter i % L), and in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(M + K + L)
    x = torch.randn(M, K, device="cuda", generator=g).abs().to(torch.bfloat16)
    a = torch.randn(L, rank, K, device="cuda", generator=g).abs().to(torch.bfloat16)
    b = torch.zeros(L, N, rank, dtype=torch.bfloat16, device="cuda")
    b[:, torch.arange(N), torch.arange(N) % rank] = 1
    ids = (torch.arange(M, device="cuda") * L // M).to(torch.int32)
    h = B.LoraLinear(torch.zeros(N, K, dtype=torch.bfloat16, device="cuda"), a, b, scale=scale, out_dtype=torch.float32)
    y = h(x, ids).double()
    s = torch.cuda.current_stream().cuda_stream
    assert B.gmmfr_check_device_errors(h._spaces[s][0], s) == 0
    want = torch.stack([x[i].double() @ a[ids[i]].double().T for i in range(M)])[:, torch.arange(N) % rank]
    return y, want if scale is None else want * scale[ids.long(), None].double()


BOUND = 32.5 * 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -21


# one adapter for all rows, or few: few CTAs have the rows, and a warp all of its CTA's K; M = 1 has no launch of its own where K is short
@pytest.mark.parametrize("M,L", [(1, 1), (2, 1), (20, 1), (32, 2), (33, 1), (100, 3), (128, 1), (128, 4), (128, 100)])
@pytest.mark.parametrize("K", [264, 2048, 7168, 16384, 40000])
def test_sums_of_few_rows(M, K, L):
    y, want = _sums(M, K, L)
    assert (y - want).norm() <= BOUND * want.norm()


@pytest.mark.parametrize("M,K,L", [(300, 328, 2), (129, 7168, 1), (1030, 4096, 40)])
def test_sums_of_many_rows(M, K, L):
    y, want = _sums(M, K, L)
    assert (y - want).norm() <= BOUND * want.norm()


@pytest.mark.parametrize("M,K,L", [(129, 16384, 1), (300, 20000, 3), (200, 40000, 1), (513, 40000, 70), (130, 200000, 2)])
def test_sums_of_many_rows_past_16384(M, K, L):
    y, want = _sums(M, K, L, scale=torch.linspace(0.5, 1.7, L, device="cuda"))
    assert (y - want).norm() <= BOUND * want.norm()


def test_bf16_results_are_one_rounding_away():
    for M, K in ((128, 40000), (300, 40000)):
        g = torch.Generator(device="cuda").manual_seed(M)
        x, a = torch.randn(M, K, device="cuda", generator=g).abs().to(torch.bfloat16), torch.rand(1, 8, K, device="cuda", generator=g).to(torch.bfloat16)
        b = torch.eye(8, dtype=torch.bfloat16, device="cuda")[None]
        y = B.LoraLinear(torch.zeros(8, K, dtype=torch.bfloat16, device="cuda"), a, b)(x, torch.zeros(M, dtype=torch.int32, device="cuda"))
        want = x.double() @ a[0].double().T
        # one accumulator may hold them all: K / 16 additions of 2^-23 at most
        assert ((y.double() - want).abs() <= (2.0 ** -8 + K / 16 * 2.0 ** -23) * want).all()
