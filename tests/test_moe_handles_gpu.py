"""The handles between calls on a GPU: refusals, graphs, streams.  Results are compared bit by bit with those of a handle
that was called once (the kernels are deterministic)."""
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


def _randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()


def _layer(E=16, H=256, I=64, topk=4):
    return B.MoeLayer(_randn(1, E, H, scale=0.1), _randn(2, E, H, 2 * I, scale=0.06), _randn(3, E, I, H, scale=0.1), topk=topk)


def test_a_good_call_after_a_refused_one():
    wide = _randn(4, 70, 260)
    x, odd = wide[:, :256].contiguous(), wide[:, :256]
    layer, gate = _layer(), B.MoeGate(_randn(1, 16, 256, scale=0.1), topk=4)
    want, want_ids = _layer()(x[:8]), B.MoeGate(_randn(1, 16, 256, scale=0.1), topk=4)(x)[0]
    for refused in (odd[:4], x[:65], odd[:40]):
        assert torch.equal(layer(x[:8]), want)
        with pytest.raises(B.GmmfrError):
            layer(refused)
        assert torch.equal(layer(x[:8]), want)
    for rows in (5, 70):
        assert torch.equal(gate(x)[0], want_ids)
        with pytest.raises(B.GmmfrError):
            gate(odd[:rows])
        assert torch.equal(gate(x)[0], want_ids)
