"""The grouped product and both gradients with the most rows that a call takes, nearly all of them one expert's: row numbers within a
few hundred of 2^31.

Rows are of -1, 0 and 1, weights whole numbers up to 8: products are at most 64, exact in BF16, and sums of all rows, random in sign,
stay far below 2^24, exact in FP32 in any order.  So results are equal, not near.
"""
import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

M, K = (1 << 31) - 1024, 8
STEP = 1 << 26  # rows at a time
FEW = 1000      # the second expert's


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 140 << 30:
        pytest.skip("takes 80 GB")
    build_mod.build()
    B.load()
    yield
    torch.cuda.empty_cache()


def _steps():
    """Rows of either expert, STEP at a time."""
    for e, begin, end in ((0, 0, M - FEW), (1, M - FEW, M)):
        for at in range(begin, end, STEP):
            yield e, slice(at, min(at + STEP, end))


def _fill(t, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for _, at in _steps():
        t[at] = torch.randint(-1, 2, t[at].shape, generator=g, device="cuda", dtype=torch.int8).to(t.dtype)


def test_most_rows():
    w = torch.randint(-8, 9, (2, 8, K), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    h = B.GroupedLinear(w, grad_dtype=torch.float32)
    groups = torch.tensor([M - FEW, FEW], device="cuda")
    x, y = (torch.empty((M, K), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = torch.cuda.current_stream().cuda_stream
    _fill(x, 2)
    for call, weight in ((h, w), (h.grad_input, w.mT)):
        y.fill_(99)
        call(x, groups, out=y)
        assert B.gmmfr_check_device_errors(h._spaces[s][0], s) == 0
        for e, at in _steps():
            assert torch.equal(y[at].float(), x[at].float() @ weight[e].float().T), (e, at)
    _fill(y, 3)
    dw = h.grad_weight(y, x, groups)
    assert B.gmmfr_check_device_errors(h._spaces[s][0], s) == 0
    want = torch.zeros((2, 8, K), dtype=torch.float64, device="cuda")
    for e, at in _steps():
        want[e] += y[at].double().T @ x[at].double()
    assert torch.equal(dw.double(), want)
