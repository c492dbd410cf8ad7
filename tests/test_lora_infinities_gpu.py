"""Both factors of an adapter infinite at one rank: the product with adapters gives what the formula gives, in kind (finite, an infinity
of its sign, or NaN), in every form."""
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


def _kind(t):
    return torch.where(t.isnan(), 3, torch.where(t.isinf(), t.sign(), 0)).to(torch.int8)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,r", [(2, 16), (16, 8), (100, 24), (128, 64), (400, 16), (520, 72)])
def test_both_factors_infinite_at_one_rank(M, r, out):
    N, K, L = 264, 328, 5
    g = torch.Generator().manual_seed(M)
    x, w, a, b = ((torch.randn(s, generator=g) * f).to(torch.bfloat16).cuda()
                  for s, f in (((M, K), 1), ((N, K), K ** -0.5), ((L, r, K), K ** -0.5), ((L, N, r), r ** -0.5)))
    x[x == 0] = 1
    ids = torch.randint(-1, L, (M,), generator=g).to(torch.int32).cuda()
    ids[:2] = 1
    inf, j = float("inf"), r - 3
    a[1, j, 9], b[1, 5, j], b[1, 263, j], b[1, 77, j], b[1, 130, j], b[1, 131, j] = inf, inf, -inf, float("nan"), 0.0, -0.0
    b[3, 40, 2], b[3, 41, 2], a[4, 1, 7] = -inf, inf, -inf  # one factor alone
    want = x.double() @ w.double().T
    for i in range(L):
        at = (ids == i).nonzero()[:, 0]
        # term by term: a matrix product of its own could take an order of its own
        s = (x[at].double()[:, None, :] * a[i].double()[None]).sum(-1)
        want[at] += (s[:, None, :] * b[i].double()[None]).sum(-1)
    y = B.LoraLinear(w, a, b, out_dtype=out)(x, ids)
    assert torch.equal(_kind(y), _kind(want))
    mine = ids == 1
    assert y[mine][:, 5].isinf().all() and (y[mine][:, 5] == -y[mine][:, 263]).all()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 20, 32, 100, 300])
@pytest.mark.parametrize("K,at", [(2056, 5), (2552, 2551), (4096, 3000)])
def test_sums_in_parts_of_which_one_is_infinite(K, at, M, out):
    """K in shares, whose parts of a sum are added by who reads them: before the products with the second factor, since
    -1 * inf + inf * inf is NaN where (-1 + inf) * inf is not."""
    N, L, r, inf = 72, 2, 8, float("inf")
    g = torch.Generator().manual_seed(K + M)
    x, w, a, b = ((torch.randn(s, generator=g) * f).to(torch.bfloat16).cuda()
                  for s, f in (((M, K), 1), ((N, K), K ** -0.5), ((L, r, K), K ** -0.5), ((L, N, r), r ** -0.5)))
    x[:, at] = x[:, at].abs() + 0.5
    ids = (torch.arange(M) % 3 - 1).to(torch.int32).cuda()
    ids[0] = 1
    a[1, 3, at], b[1, 4, 3], b[1, 71, 3], b[1, 30, 3] = inf, inf, -inf, 0.0
    y = B.LoraLinear(w, a, b, out_dtype=out)(x, ids)
    mine = ids == 1
    assert (y[mine][:, 4] == inf).all() and (y[mine][:, 71] == -inf).all() and y[mine][:, 30].isnan().all()
    rest = [n for n in range(N) if n not in (4, 30, 71)]
    assert (y[mine][:, rest] == b[1, rest, 3].float().sign()[None] * inf).all() and y[~mine].isfinite().all()
