"""GPU parity of the dense product with adapters against a float64 oracle.

Tolerances, from the arithmetic: a tensor core adds 16 products at a time to the running sum and may truncate, K/16
additions of at most 2^-23 relative each; K/8 * 2^-23 * sum |x w| leaves a factor of two, and holds for x A^T alike.  The
products with B are FP32 additions, rank * 2^-23 of their terms' sum; the sums of rows of x with A enter them in whole, or for
BF16 results as two BF16 numbers, off by 2^-17 of each sum at most: K/8 * 2^-23 + 2^-17 + rank * 2^-23 of the adapters' terms in
all, without the 2^-17 for FP32 results, whose three numbers may be added in 3 rank / 16 steps each: 3 rank / 8 * 2^-23.  An
activation evaluated with the approximate exponential and division is a few 2^-22 off, taken as 2^-20 of its value.  BF16
results are rounded once, 2^-9 relative; 2^-8 allows for a neighbour.
"""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod
from oracle import grouped as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.load()


def _randn(seed, *shape, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _bits(handle):
    s = torch.cuda.current_stream().cuda_stream
    return B.gmmfr_check_device_errors(handle._spaces[s][0], s)


def _ids(M, L, kind, seed=3):
    g = torch.Generator().manual_seed(seed)
    if kind == "none":
        return torch.full((M,), -1, dtype=torch.int32).cuda()
    if kind == "one":
        return torch.full((M,), L - 1, dtype=torch.int32).cuda()
    ids = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    if kind == "runs":
        at = 0
        while at < M:
            n = int(torch.randint(1, M // 3 + 2, (1,), generator=g))
            ids[at:at + n] = ids[at].clone()
            at += n
    return ids.cuda()


def _case(M, N, K, L, r, act="none", bias=False, residual=False, out=torch.bfloat16, ids="tokens"):
    rows = 2 * N if act == "swiglu" else N
    x, w = _randn(1, M, K), _randn(2, rows, K, scale=K ** -0.5)
    a, b = _randn(4, L, r, K, scale=K ** -0.5), _randn(5, L, rows, r, scale=r ** -0.5)
    scale = torch.linspace(0.5, 2.0, L, device="cuda")
    bt = _randn(6, rows, scale=0.3) if bias else None
    res = _randn(7, M, N) if residual else None
    id_t = _ids(M, L, ids)
    h = B.LoraLinear(w, a, b, scale=scale, bias=bt, activation=act, out_dtype=out)
    y = h(x, id_t, residual=res)
    assert _bits(h) == 0
    ref, absb = O.lora_linear(_f64(x), _f64(w), _f64(a), _f64(b), _f64(scale), id_t.cpu().numpy(), _f64(bt), _f64(res), act)
    split = 2.0 ** -17 * (ids != "none" and out == torch.bfloat16)
    tol = (max(K, 16) / 8 * 2.0 ** -23 + split + r * 2.0 ** -23) * absb + 2.0 ** -20 * np.abs(ref)
    if out == torch.bfloat16:
        tol += 2.0 ** -8 * np.abs(ref)
    err = np.abs(_f64(y) - ref)
    assert np.all(err <= tol), (float(err.max()), float((err / (tol + 1e-30)).max()))
    return h, x, id_t, res, y


# rows, N, K, adapters, rank: every form of the product, and both tiles of the sums
SIZES = [(1, 64, 64, 1, 8), (1, 2048, 2048, 64, 16), (3, 40, 72, 5, 8), (8, 200, 520, 3, 24), (13, 512, 1032, 40, 16), (17, 96, 256, 7, 40),
         (32, 300, 512, 9, 32), (33, 4096, 2048, 20, 16), (64, 1000, 4096, 70, 64), (100, 264, 1288, 6, 128), (128, 777, 640, 200, 16),
         (129, 320, 264, 4, 16), (200, 1024, 512, 33, 8), (257, 512, 1096, 2, 72), (300, 136, 2048, 11, 256), (777, 1285, 328, 32, 32),
         (1030, 4096, 2048, 5, 16)]


@pytest.mark.parametrize("ids", ["tokens", "runs"])
@pytest.mark.parametrize("M,N,K,L,r", SIZES)
def test_product_with_adapters(M, N, K, L, r, ids):
    _case(M, N, K, L, r, ids=ids)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("M,N,K,L,r", [(5, 72, 136, 3, 16), (24, 2048, 1024, 8, 16), (70, 200, 328, 12, 24), (300, 328, 512, 9, 48)])
def test_activations(M, N, K, L, r, act):
    _case(M, N, K, L, r, act=act, bias=True, residual=True)


@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
@pytest.mark.parametrize("M,N,K,L,r", [(5, 72, 136, 3, 16), (70, 200, 3336, 12, 24), (300, 328, 2056, 9, 48), (1030, 200, 512, 40, 16)])
def test_float32_results(M, N, K, L, r, act):
    _case(M, N, K, L, r, act=act, bias=True, residual=True, out=torch.float32)


@pytest.mark.parametrize("M", [1, 20, 100, 600])
@pytest.mark.parametrize("ids", ["none", "one"])
def test_no_row_and_every_row_with_one_adapter(M, ids):
    _case(M, 264, 512, 7, 16, ids=ids)


@pytest.mark.parametrize("M", [1, 20, 100, 600])
def test_without_adapters_it_is_the_dense_product(M):
    x, w, bias, res = _randn(1, M, 520), _randn(2, 264, 520, scale=0.05), _randn(3, 264), _randn(4, M, 264)
    a, b = torch.full((2, 16, 520), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.full((2, 264, 16), float("inf"),
                                                                                                 dtype=torch.bfloat16, device="cuda")
    y = B.LoraLinear(w, a, b, bias=bias, activation="silu")(x, _ids(M, 2, "none"), residual=res)
    assert torch.equal(y, B.Linear(w, bias=bias, activation="silu")(x, residual=res))


@pytest.mark.parametrize("M", [16, 100, 400])
def test_what_is_not_finite_reaches_its_own_rows(M):
    N, K, L, r = 200, 328, 6, 16
    x, w = _randn(1, M, K), _randn(2, N, K, scale=K ** -0.5)
    a, b = _randn(4, L, r, K, scale=K ** -0.5), _randn(5, L, N, r, scale=r ** -0.5)
    ids = _ids(M, L, "tokens")
    want = B.LoraLinear(w, a, b)(x, ids)
    bad_a, bad_b, bad_x = a.clone(), b.clone(), x.clone()
    bad_a[2, 5, 7], bad_b[4, 10, 3], bad_x[M // 2, 9] = float("nan"), float("inf"), float("inf")
    y = B.LoraLinear(w, bad_a, bad_b)(bad_x, ids)
    hurt = (ids == 2) | (ids == 4)
    hurt[M // 2] = True
    assert torch.equal(y[~hurt], want[~hurt])
    assert not y[ids == 2].isfinite().any() and not y[ids == 4][:, 10].isfinite().any() and not y[M // 2].isfinite().any()
    rest = [n for n in range(N) if n != 10]
    at = (ids == 4) & (torch.arange(M, device="cuda") != M // 2)
    assert torch.equal(y[at][:, rest], want[at][:, rest])


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("M,N,K,r", [(40, 1032, 2048, 24), (128, 300, 4096, 64), (130, 264, 136, 8), (513, 1096, 1288, 40)])
def test_one_number_of_a_factor_that_is_not_finite(M, N, K, r, act, out):
    # wherever it lies, all else is as with a zero in its place, and its own sum with the rows' other products
    L, rows = 9, 2 * N if act == "swiglu" else N
    x, w = _randn(1, M, K), _randn(2, rows, K, scale=K ** -0.5)
    a, b = _randn(4, L, r, K, scale=K ** -0.5), _randn(5, L, rows, r, scale=r ** -0.5)
    ids = _ids(M, L, "tokens")
    for adapter, row, j, bad in [(0, 0, 0, "nan"), (8, rows - 1, r - 1, "inf"), (4, 33, r // 2, "-inf"), (7, rows // 2 + 70, 7, "nan")]:
        b0, b1 = b.clone(), b.clone()
        b0[adapter, row, j], b1[adapter, row, j] = 0, float(bad)
        zero, y = (B.LoraLinear(w, a, f, activation=act, out_dtype=out)(x, ids) for f in (b0, b1))
        its = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        its[ids == adapter, row % N] = True
        assert its.any() and torch.equal(y[~its], zero[~its])
        if act == "none":
            assert not y[its].isfinite().any()


def test_strided_weight():
    M, N, K = 300, 136, 200
    x, w, ids = _randn(1, M, K), _randn(2, N, 264), _ids(M, 5, "tokens")
    a, b = _randn(4, 5, 16, K, scale=K ** -0.5), _randn(5, 5, N, 16)
    for m in (1, 20, 100, M):
        assert torch.equal(B.LoraLinear(w[:, :K], a, b)(x[:m], ids[:m]), B.LoraLinear(w[:, :K].contiguous(), a, b)(x[:m], ids[:m]))


@pytest.mark.parametrize("M", [4, 100, 400])
def test_an_adapter_that_there_is_not_counts_as_none_and_is_reported(M):
    N, K, L, r = 72, 136, 3, 8
    x, w = _randn(1, M, K), _randn(2, N, K)
    h = B.LoraLinear(w, _randn(4, L, r, K), _randn(5, L, N, r))
    ids = _ids(M, L, "tokens")
    good = ids.clone()
    ids[0], ids[M // 2], ids[M - 1] = -2, 3, 1 << 30
    good[0] = good[M // 2] = good[M - 1] = -1
    y = h(x, ids)
    assert _bits(h) == B.DEV_BAD_ADAPTER_ID
    assert torch.equal(y, h(x, good)) and _bits(h) == 0


def test_strides():
    M, N, K = 40, 136, 200
    h, x, ids, res, y = _case(M, N, K, 5, 16, residual=True)
    wide = _randn(8, M, 264)
    wide[:, 8:208] = x
    wide_res = _randn(9, M, 139)
    wide_res[:, 1:137] = res
    out = torch.full((M, 139), 5.0, dtype=torch.bfloat16, device="cuda")
    h(wide[:, 8:208], ids, residual=wide_res[:, 1:137], out=out[:, 2:138])
    assert torch.equal(out[:, 2:138], y) and (out[:, :2] == 5).all() and (out[:, 138:] == 5).all()
    assert torch.equal(h(x, ids, residual=res, out=res), y) and torch.equal(res, y)  # in the residual's place


@pytest.mark.parametrize("M", [5, 100, 700])
def test_other_streams_and_captured_graphs(M):
    h, x, ids, res, y = _case(M, 264, 512, 9, 16, residual=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = h(x, ids, residual=res, stream=s)
    s.synchronize()
    assert torch.equal(got, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = h(x, ids, residual=res)
        again = h(out[:, :264].new_zeros(M, 512), ids, residual=out)  # a second call behind the first, in the same workspace
    # other rows, adapters and factors in the same memory
    ids.copy_(_ids(M, 9, "tokens", seed=11)), x.copy_(_randn(12, M, 512)), h._keep[1].copy_(_randn(13, 9, 16, 512, scale=0.05))
    h._keep[2].copy_(_randn(14, 9, 264, 16))
    want = h(x, ids, residual=res)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(again, want)


def test_calls_one_after_the_other_share_a_workspace():
    """Sums of one call are not overwritten by the next's, nor read before they are there, over many sizes back to back."""
    N, K, L, r = 520, 1024, 16, 16
    w, a, b = _randn(2, N, K, scale=0.03), _randn(4, L, r, K, scale=0.03), _randn(5, L, N, r)
    h = B.LoraLinear(w, a, b)
    sizes = [1, 40, 8, 300, 128, 2, 77, 1030, 16] * 4
    xs = [_randn(20 + i, M, K) for i, M in enumerate(sizes)]
    ids = [_ids(M, L, "tokens", seed=50 + i) for i, M in enumerate(sizes)]
    ys = [h(x, i) for x, i in zip(xs, ids)]
    torch.cuda.synchronize()
    for x, i, y in zip(xs, ids, ys):
        assert torch.equal(h(x, i), y)
        torch.cuda.synchronize()


@pytest.mark.parametrize("M", [3, 50, 300])
def test_offsets_past_32_bits(M):
    """Second factors, and first ones, of more than 2^31 elements each: the last adapter is read where it lies."""
    N, K, r, L = 4096, 4096, 64, 8200
    x, w = _randn(1, M, K), _randn(2, N, K, scale=K ** -0.5)
    a1, b1 = _randn(3, 1, r, K, scale=K ** -0.5), _randn(4, 1, N, r, scale=r ** -0.5)
    a, b = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((L, r, K), (L, N, r)))
    a[-1], b[-1] = a1[0], b1[0]
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[::2] = L - 1
    f32 = dict(out_dtype=torch.float32)
    want, got = B.LoraLinear(w, a1, b1, **f32)(x, torch.where(ids < 0, ids, 0)), B.LoraLinear(w, a, b, **f32)(x, ids)
    # the number of adapters shares the sums out in another way: each is within K/8 * 2^-23 of the terms' sum, 2^-17 of the
    # adapters' (above), of the value
    mine = (ids >= 0)[:, None]
    terms, more = x.abs().float() @ w.abs().float().T, (x.abs().float() @ a1[0].abs().float().T) @ b1[0].abs().float().T * mine
    assert ((got - want).abs() <= 2 * (K / 8 * 2 ** -23 * (terms + more) + (2 ** -17 + r * 2 ** -23) * more)).all()
    assert torch.equal(got[1::2], want[1::2]) and (got - B.Linear(w, **f32)(x))[::2].abs().max() > 0.1


def test_a_step_of_a_block_with_adapters():
    """Router, routed experts as grouped products, and a shared expert with adapters beside them, as one step of a served
    model, against the formula in 64 bits."""
    T, H, I, E, k, L, r = 70, 256, 128, 8, 2, 5, 16
    x, wg = _randn(1, T, H), _randn(2, E, H, scale=0.2)
    w13, w2 = _randn(3, E, 2 * I, H, scale=H ** -0.5), _randn(4, E, H, I, scale=I ** -0.5)
    s13, s2 = _randn(5, 2 * I, H, scale=H ** -0.5), _randn(6, H, I, scale=I ** -0.5)
    a13, b13 = _randn(7, L, r, H, scale=H ** -0.5), _randn(8, L, 2 * I, r, scale=r ** -0.5)
    a2, b2 = _randn(9, L, r, I, scale=I ** -0.5), _randn(10, L, H, r, scale=r ** -0.5)
    ids = _ids(T, L, "tokens")
    experts, weights = B.MoeGate(wg, topk=k)(x)
    routed, _ = B.route(experts, weights, x.view(torch.uint8), torch.empty((T, 2 * H // 64, 2), dtype=torch.uint8, device="cuda"), E)
    rows, groups, perm = routed["x1"].view(torch.bfloat16), routed["group_list"], routed["perm"].long()
    up = B.GroupedLinear(w13, out_dtype=torch.float32)(rows, groups)
    mid = (torch.nn.functional.silu(up[:, :I]) * up[:, I:]).to(torch.bfloat16)
    down = B.GroupedLinear(w2, out_dtype=torch.float32)(mid, groups)
    shared = B.LoraLinear(s13, a13, b13, activation="swiglu")(x, ids)
    out = B.LoraLinear(s2, a2, b2, out_dtype=torch.float32)(shared, ids, residual=x)
    out = out.index_add(0, perm // k, down * weights.flatten()[perm, None])
    ref = x.double()
    w13d, w2d = w13.double(), w2.double()
    for j in range(k):
        z = torch.einsum("th,tnh->tn", x.double(), w13d[experts[:, j].long()])
        z = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
        ref = ref + weights[:, j, None].double() * torch.einsum("ti,thi->th", z, w2d[experts[:, j].long()])
    adapter = [torch.where((ids >= 0)[:, None, None], t.double()[ids.clamp(min=0).long()], 0.0) for t in (a13, b13, a2, b2)]
    z = x.double() @ s13.double().T + torch.einsum("tnr,trh,th->tn", adapter[1], adapter[0], x.double())
    z = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
    ref = ref + z @ s2.double().T + torch.einsum("tnr,tri,ti->tn", adapter[3], adapter[2], z)
    # two roundings to BF16 on the way, of the experts' and of the shared expert's middle: 2^-9 of terms that add up at random
    assert float((out.double() - ref).norm() / ref.norm()) < 2 ** -8
