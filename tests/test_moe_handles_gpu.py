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


def _busy(*sizes):
    """Gives back to the current stream's pool blocks of these bytes that the stream still writes to; what is returned
    lies between them and keeps them from growing together; and the addresses."""
    torch.cuda.synchronize()
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(128)]
    torch.cuda._sleep(200_000_000)
    for b in blocks:
        b.fill_(255)
    return blocks[::2], {b.data_ptr() for b in blocks[1::2]}


def test_outputs_on_another_stream_take_no_memory_that_this_one_still_writes_to():
    x, w = _randn(8, 2000, 256), _randn(9, 16, 256, scale=0.1)
    gate, lin, layer, s = B.MoeGate(w, topk=4), B.Linear(w), _layer(), torch.cuda.Stream()
    ids, weights = gate(x)
    y, out = lin(x), layer(x[:9])
    between, used = _busy(ids.nbytes, y.nbytes, out.nbytes)
    got = (*gate(x, stream=s), lin(x, stream=s), layer(x[:9], stream=s))
    assert not used & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    del between
    for a, b in zip(got, (ids, weights, y, out)):
        assert torch.equal(a, b)


def test_functions_on_another_stream_take_no_memory_that_this_one_still_writes_to():
    s = torch.cuda.Stream()
    E, H, I, N = 4, 256, 64, 300
    w13, w2, x = _randn(2, E, H, 2 * I, scale=0.06), _randn(3, E, I, H, scale=0.1), _randn(4, N, H)
    ends = torch.tensor([0, 100, 100, 250, 300], dtype=torch.int32, device="cuda")
    prepared = B.ffn_prepare(H, I, E, w13, w2)
    want, _ = B.ffn(x, prepared, ends, H, I, E)
    codes = [torch.randint(0, 120, shape, dtype=torch.uint8, device="cuda") for shape in ((E, H, 2 * I), (E, I, H))]
    scales = [torch.full((E, k, n, 2), 120, dtype=torch.uint8, device="cuda") for k, n in ((H // 64, 2 * I), (I // 64, H))]
    mx = B.ffn_prepare_mx(H, I, E, codes[0], scales[0], codes[1], scales[1])
    ids = torch.randint(0, E, (N, 2), dtype=torch.int32, device="cuda")
    wt, tok_scale = torch.rand(N, 2, device="cuda"), torch.full((N, H // 64, 2), 127, dtype=torch.uint8, device="cuda")
    routed, _ = B.route(ids, wt, x.view(torch.uint8)[:, :H].contiguous(), tok_scale, E)
    few = x.view(torch.uint8)[:, :H].contiguous()
    between, used = _busy(prepared.nbytes, want.nbytes, mx.nbytes, *(t.nbytes for t in routed.values()))
    got = B.ffn_prepare(H, I, E, w13, w2, stream=s)
    got_mx = B.ffn_prepare_mx(H, I, E, codes[0], scales[0], codes[1], scales[1], stream=s)
    got_routed, ws = B.route(ids, wt, few, tok_scale, E, stream=s)
    y, ws2 = B.ffn(x, got, ends, H, I, E, stream=s)
    assert not used & {t.data_ptr() for t in (got, got_mx, y, ws, ws2, *got_routed.values())}
    torch.cuda.synchronize()
    del between
    assert torch.equal(got, prepared) and torch.equal(got_mx, mx) and torch.equal(y, want)
    for k in routed:
        assert torch.equal(got_routed[k], routed[k])


def test_a_handle_dropped_while_another_stream_uses_its_weights():
    x, s = _randn(10, 8, 256), torch.cuda.Stream()
    want = _layer()(x)
    layer = _layer()
    layer(x)
    torch.cuda.synchronize()
    size = layer.prepared.numel()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    out = layer(x, stream=s)
    del layer
    taken = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all((t == 255).all() for t in taken)


def test_first_calls_inside_a_capture_and_streams_by_address():
    """A handle whose first call on a stream is a captured one, dropped before the next capture; and any object that has a
    stream's address as a stream."""
    x = _randn(11, 20, 256)
    layer, gate, lin = _layer(), B.MoeGate(_randn(1, 16, 256, scale=0.1), topk=4), B.Linear(_randn(5, 48, 256))
    want = layer(x), gate(x)[1], lin(x)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        fresh = _layer(), B.MoeGate(_randn(1, 16, 256, scale=0.1), topk=4), B.Linear(_randn(5, 48, 256))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = fresh[0](x), fresh[1](x)[1], fresh[2](x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        del fresh, graph, out

    class Address:
        cuda_stream = stream.cuda_stream

    ids = torch.zeros((20, 1), dtype=torch.int32, device="cuda")
    codes = x.view(torch.uint8)
    scale = torch.full((20, 8, 2), 127, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got, _ = B.route(ids, torch.ones((20, 1), device="cuda"), codes, scale, 4, stream=Address)
    torch.cuda.synchronize()
    assert torch.equal(got["x1"], codes)
