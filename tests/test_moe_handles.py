"""The handles' own bookkeeping, on the host: real library checks, tensors that are addresses only, and a recording
function in place of the C entry.  (No GPU: nothing is launched and no address is read.)"""
import gc
import weakref

import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    return B.load()


class FakeTensor:
    """What the handles ask of a 2-D device tensor."""
    _next = 1 << 20

    def __init__(self, *shape, dtype=torch.bfloat16, ld=None, device=0, off=0):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.ld = shape[1] if ld is None else ld
        self.index = device
        FakeTensor._next += 1 << 20
        self.address = FakeTensor._next + off
        self.streams = []

    is_cuda = True
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.ld, 1)

    def is_contiguous(self):
        return self.shape[0] <= 1 or self.ld == self.shape[1]

    def data_ptr(self):
        return self.address

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def element_size(self):
        return self.dtype.itemsize

    def record_stream(self, stream):
        self.streams.append(stream)


class Calls:
    """A C entry's place: runs the real entry's checks as far as `status` says, and keeps the problem it was given."""

    def __init__(self, handle):
        self.handle, self.problems, self.workspaces = handle, [], []
        handle._fn = self

    def __call__(self, ref, *args):
        p = self.handle._p
        self.problems.append(type(p).from_buffer_copy(p))
        self.workspaces.append((args[-3].value, args[-2].value))
        return 0


@pytest.fixture
def fakes(monkeypatch):
    def init(self, device):
        self._lib, self._device, self._index = B.load(), torch.device("cuda", 0), 0
        self._raw_stream = lambda index: 7
        self._current = lambda: 0
        self._spaces, self._outgrown = {}, []

    monkeypatch.setattr(B._Handle, "__init__", init)
    monkeypatch.setattr(B._Handle, "_new", lambda self, shape, dtype, stream: FakeTensor(*shape, dtype=dtype))
    spaces = []

    def space(nbytes, dtype, device):
        spaces.append(FakeTensor(1, nbytes, dtype=dtype))
        return spaces[-1]

    monkeypatch.setattr(torch, "empty", space)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    prepared = FakeTensor(1, 1 << 20, dtype=torch.uint8)
    monkeypatch.setattr(B.MoeLayer, "_prepare", staticmethod(lambda *a: prepared))
    return spaces


def _gate(**kw):
    g = B.MoeGate(FakeTensor(64, 128), topk=4, **kw)
    return g, Calls(g)


def _layer(**kw):
    w2 = type("W", (), {"shape": (16, 64, 128)})()
    h = B.MoeLayer(FakeTensor(16, 128), None, w2, topk=4, **kw)
    return h, Calls(h)


# ------------------------------------------------------------------------- a refused call leaves nothing behind
@pytest.mark.parametrize("refused", [50, 1000])
def test_gate_runs_the_rows_it_is_given_after_a_refused_call(fakes, refused):
    gate, calls = _gate()
    gate(FakeTensor(100, 128))
    with pytest.raises(B.GmmfrError):
        gate(FakeTensor(refused, 128, ld=132))  # rows off 16-byte boundaries
    ids, weights = gate(FakeTensor(100, 128))
    assert [p.T for p in calls.problems] == [100, 100] and calls.problems[-1].ldx == 0
    assert ids.shape == weights.shape == (100, 4)


@pytest.mark.parametrize("refused,ld", [(4, 132), (40, 132), (65, 128)])
def test_layer_runs_the_rows_it_is_given_after_a_refused_call(fakes, refused, ld):
    layer, calls = _layer()

    def entry(ref, *args):
        # the real entry's refusals come from the same check
        B.gmmfr_moe_layer_workspace_size(layer._p)
        return calls(ref, *args)

    layer._fn = entry
    layer(FakeTensor(8, 128))
    with pytest.raises(B.GmmfrError):
        layer(FakeTensor(refused, 128, ld=ld))
    out = layer(FakeTensor(8, 128))
    assert [p.gate.T for p in calls.problems] == [8, 8] and out.shape == (8, 128)


def test_linear_runs_the_rows_it_is_given_after_a_refused_call(fakes):
    lin = B.Linear(FakeTensor(16, 128))
    calls = Calls(lin)
    lin(FakeTensor(8, 128))
    with pytest.raises(B.GmmfrError):
        lin(FakeTensor(1 << 31, 128))
    lin(FakeTensor(8, 128))
    assert [p.M for p in calls.problems] == [8, 8]


def test_a_stride_of_one_call_is_not_the_next_ones(fakes):
    layer, calls = _layer()
    layer(FakeTensor(8, 128), residual=FakeTensor(8, 128, ld=131), out=FakeTensor(8, 128, ld=133))
    layer(FakeTensor(8, 128))
    assert [(p.ld_residual, p.ld_out) for p in calls.problems] == [(131, 133), (0, 0)]
    lin = B.Linear(FakeTensor(16, 128))
    calls = Calls(lin)
    lin(FakeTensor(8, 128), residual=FakeTensor(8, 16, ld=19), out=FakeTensor(8, 16, ld=17))
    lin(FakeTensor(8, 128))
    assert [(p.ld_residual, p.ld_out) for p in calls.problems] == [(19, 17), (0, 0)]


# ------------------------------------------------------------------------- what a captured graph writes to stays
def test_every_number_of_tokens_takes_the_same_layer_workspace(fakes):
    layer, calls = _layer()
    for T in (1, 16, 64, 3):
        layer(FakeTensor(T, 128))
    assert len({w[0] for w in calls.workspaces}) == 1
    layer._p.gate.T = 64
    assert calls.workspaces[0][1] >= B.gmmfr_moe_layer_workspace_size(layer._p)


def test_an_outgrown_workspace_stays_with_the_handle(fakes):
    lin = B.Linear(FakeTensor(16, 129))  # rows off 16-byte boundaries: copies, whose size goes with the rows
    calls = Calls(lin)
    for M in (64, 128, 4096, 5000, 100000):
        lin(FakeTensor(M, 129))
        assert calls.workspaces[-1][1] >= B.gmmfr_linear_workspace_size(lin._p)
    kept = [weakref.ref(t) for t in fakes]
    addresses = [t.address for t in fakes]
    largest = fakes[-1].numel()
    assert len(fakes) > 2 and sum(t.numel() for t in fakes[:-1]) < largest + 256
    fakes.clear()
    gc.collect()
    assert all(r() is not None for r in kept)
    assert {w[0] for w in calls.workspaces} <= set(addresses)
    del lin, calls
    gc.collect()
    assert not any(r() is not None for r in kept)
