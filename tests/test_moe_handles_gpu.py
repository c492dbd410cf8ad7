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


def test_graphs_of_growing_sizes_captured_on_one_stream():
    """Each size warmed up and captured in turn; whatever memory the handles gave back is taken and watched while the
    graphs are replayed."""
    layer = _layer()
    lin = B.Linear(_randn(5, 48, 129))
    x, y = _randn(6, 64, 256), _randn(7, 4096, 129)
    sizes, rows = (1, 16, 64), (40, 700, 4096)
    want = [(_layer()(x[:T]), B.Linear(_randn(5, 48, 129))(y[:M])) for T, M in zip(sizes, rows)]
    stream, graphs = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for T, M in zip(sizes, rows):
            layer(x[:T]), lin(y[:M])
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                out = layer(x[:T]), lin(y[:M])
            graphs.append((graph, out))
        layer(x), lin(y)
        taken = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in (1 << 10, 1 << 13, 1 << 16, 1 << 19, 1 << 21, 1 << 22)
                 for _ in range(20)]
    torch.cuda.synchronize()
    for _ in range(2):
        for (graph, out), ref in zip(graphs, want):
            for o in out:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert all((t == 77).all() for t in taken)
