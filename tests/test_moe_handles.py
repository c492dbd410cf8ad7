"""The handles' own bookkeeping, on the host: real library checks, tensors that are addresses only, and a recording
function in place of the C entry.  (No GPU: nothing is launched and no address is read.)"""
import contextlib
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
        self.ld = shape[-1] if ld is None else ld
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
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    prepared = FakeTensor(1, 1 << 20, dtype=torch.uint8)
    monkeypatch.setattr(B.MoeLayer, "_prepare", staticmethod(lambda *a: prepared))
    return spaces


def _gate(**kw):
    g = B.MoeGate(FakeTensor(64, 128), topk=4, **kw)
    return g, Calls(g)


def _layer(**kw):
    h = B.MoeLayer(FakeTensor(16, 128), FakeTensor(16, 128, 128), FakeTensor(16, 64, 128), topk=4, **kw)
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


# ------------------------------------------------------------------------- devices
def test_tensors_of_another_device_are_refused(fakes):
    gate, gate_calls = _gate()
    layer, layer_calls = _layer()
    lin = B.Linear(FakeTensor(16, 128))
    lin_calls = Calls(lin)
    here, there = FakeTensor(8, 128), FakeTensor(8, 128, device=1)
    host = FakeTensor(8, 128, device=-1)
    i32 = dict(dtype=torch.int32, device=1)
    f32 = dict(dtype=torch.float32, device=1)
    for call in (lambda: gate(there), lambda: layer(there), lambda: lin(there), lambda: gate(host), lambda: lin(host),
                 lambda: gate(here, ids=FakeTensor(8, 4, **i32)), lambda: gate(here, weights=FakeTensor(8, 4, **f32)),
                 lambda: gate(here, logits=FakeTensor(8, 64, **f32)), lambda: layer(here, residual=there),
                 lambda: layer(here, out=there), lambda: layer(here, topk_ids=FakeTensor(8, 4, **i32)),
                 lambda: layer(here, topk_weights=FakeTensor(8, 4, **f32)),
                 lambda: lin(here, residual=FakeTensor(8, 16, device=1)), lambda: lin(here, out=FakeTensor(8, 16, device=1)),
                 lambda: B.MoeGate(FakeTensor(64, 128, device=1), topk=2),
                 lambda: B.Linear(FakeTensor(16, 128), bias=FakeTensor(16, device=1)),
                 lambda: B.MoeLayer(FakeTensor(16, 128), FakeTensor(16, 128, 128, device=1), FakeTensor(16, 64, 128), topk=2)):
        with pytest.raises(ValueError, match="cuda:1|device tensors"):
            call()
    assert not gate_calls.problems and not layer_calls.problems and not lin_calls.problems


def test_a_call_runs_on_the_device_of_its_handle(fakes, monkeypatch):
    current = [1]

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    seen = []
    for handle, x in ((_gate()[0], FakeTensor(8, 128)), (_layer()[0], FakeTensor(8, 128)), (B.Linear(FakeTensor(16, 128)), FakeTensor(8, 128))):
        handle._current = lambda: current[0]
        handle._fn = lambda *a: seen.append(current[0]) or 0
        handle(x)
    assert seen == [0, 0, 0] and current == [1]


# ------------------------------------------------------------------------- weights of the wrong kind
def _mx_weights(**kw):
    E, H, I = 4, 128, 64
    u8 = dict(dtype=torch.uint8)
    w = dict(w13=FakeTensor(E, H, 2 * I, dtype=torch.float8_e4m3fn), w13_scale=FakeTensor(E, H // 64, 2 * I, 2, **u8),
             w2=FakeTensor(E, I, H, **u8), w2_scale=FakeTensor(E, I // 64, H, 2, **u8))
    w.update(kw)
    return (H, I, E), w


@pytest.mark.parametrize("bad", [
    dict(w13=FakeTensor(4, 128, 128, dtype=torch.float8_e5m2)), dict(w2=FakeTensor(4, 64, 128, dtype=torch.bool)),
    dict(w2=FakeTensor(4, 64, 128, dtype=torch.float8_e5m2)), dict(w2_scale=FakeTensor(4, 1, 128, 2, dtype=torch.float8_e4m3fn)),
    dict(w13_scale=FakeTensor(4, 2, 128, 2, dtype=torch.float8_e5m2)), dict(w13_scale=FakeTensor(4, 2, 64, 2, dtype=torch.uint8)),
    dict(w2_scale=None), dict(w13=FakeTensor(4, 128, 128))], ids=lambda b: next(iter(b)))
def test_mx_weights_of_another_type_are_refused(bad):
    (H, I, E), w = _mx_weights(**bad)
    with pytest.raises(ValueError, match=next(iter(bad))):
        B.ffn_prepare_mx(H, I, E, w["w13"], w["w13_scale"], w["w2"], w["w2_scale"])


def test_layers_with_half_of_their_weights_are_refused(monkeypatch):
    def init(self, device):
        self._device, self._index = torch.device("cuda", 0), 0

    monkeypatch.setattr(B._Handle, "__init__", init)
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    _, w = _mx_weights()
    gate = FakeTensor(4, 128)
    bf16 = dict(w13=FakeTensor(4, 128, 128), w2=FakeTensor(4, 64, 128))
    monkeypatch.setattr(B, "ffn_prepare", lambda *a: FakeTensor(1, 1 << 20, dtype=torch.uint8))
    for kw in ({**w, "w2_scale": None}, {**w, "w13_scale": None}, {**bf16, "w2_scale": w["w2_scale"]},
               {**bf16, "shared_w13": FakeTensor(128, 128)}, {**bf16, "shared_w2": FakeTensor(64, 128)},
               {**bf16, "w13": w["w13"]}):
        with pytest.raises(ValueError):
            B.MoeLayer(gate, topk=2, **kw)
