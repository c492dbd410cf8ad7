"""GPU parity of the products grouped by expert, and of their gradients, against float64 oracles.

Tolerances, from the arithmetic: a tensor core adds 16 products at a time to the running sum and may truncate, K/16
additions of at most 2^-23 relative each; K/8 * 2^-23 * sum |w x| leaves a factor of two.  FP32 results besides add up to
K/1024 such sums to nearest, less than what the factor leaves.  BF16 results are rounded once, 2^-9 relative; 2^-8 allows for a
neighbour.  Sums of rows shorter than 16 still take one addition, so K counts as 16 at least.
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


def _randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()


def _f64(t):
    return t.detach().cpu().double().numpy()


def _close(got, ref, absb, terms, what):
    tol = max(np.max(terms), 16) / 8 * 2.0 ** -23 * absb + (2.0 ** -8 * np.abs(ref) if got.dtype == torch.bfloat16 else 0)
    err = np.abs(_f64(got) - ref)
    assert np.all(err <= tol), (what, float(err.max()), float((err / (tol + 1e-30)).max()))


def _list(sizes, kind):
    t = torch.tensor(sizes, dtype=torch.int64)
    return (t if kind == 1 else t.cumsum(0)).cuda()


def _bits(handle):
    s = torch.cuda.current_stream().cuda_stream
    return B.gmmfr_check_device_errors(handle._spaces[s][0], s)


# rows of each expert, rows behind the last, N, K
SIZES = [
    ([1], 0, 8, 8),
    ([3], 2, 64, 64),
    ([5, 0, 1, 17, 2], 0, 72, 136),
    ([0, 0, 40, 0], 5, 264, 64),
    ([33, 64, 31, 32], 1, 256, 128),
    ([65, 0, 100, 3, 128], 0, 520, 200),
    ([129, 256, 1, 255, 7], 3, 384, 320),
    ([257, 15, 300, 16], 0, 256, 1096),
    ([700, 0, 513], 40, 136, 2112),
    ([2] * 300, 0, 96, 96),
    ([1, 0] * 500, 0, 40, 72),
]
IDS = [f"E{len(s)}_M{sum(s) + r}_N{n}_K{k}" for s, r, n, k in SIZES]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("sizes,rest,N,K", SIZES, ids=IDS)
def test_product(sizes, rest, N, K, transposed, out):
    E, M = len(sizes), sum(sizes) + rest
    x, w = _randn(1, M, K), _randn(2, E, N, K, scale=K ** -0.5)
    h = B.GroupedLinear(w.mT.contiguous() if transposed else w, transposed=transposed, out_dtype=out)
    y = h(x, _list(sizes, 1))
    assert _bits(h) == 0
    ref, absb = O.grouped_linear(_f64(x), _f64(w), sizes)
    _close(y, ref, absb, K, "y")
    assert not y[M - rest:].any()


@pytest.mark.parametrize("transposed", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("sizes,rest,N,K", SIZES, ids=IDS)
def test_rows_gradient(sizes, rest, N, K, transposed):
    E, M = len(sizes), sum(sizes) + rest
    dy, w = _randn(1, M, N), _randn(2, E, N, K, scale=N ** -0.5)
    h = B.GroupedLinear(w.mT.contiguous() if transposed else w, transposed=transposed, group_list_type=0)
    dx = h.grad_input(dy, _list(sizes, 0))
    assert _bits(h) == 0
    ref, absb = O.grouped_linear(_f64(dy), _f64(w).transpose(0, 2, 1), sizes)
    _close(dx, ref, absb, N, "dx")
    assert not dx[M - rest:].any()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("sizes,rest,N,K", SIZES, ids=IDS)
def test_weights_gradient(sizes, rest, N, K, transposed, out):
    E, M = len(sizes), sum(sizes) + rest
    x, dy, w = _randn(1, M, K), _randn(2, M, N), _randn(3, E, N, K)
    h = B.GroupedLinear(w.mT.contiguous() if transposed else w, transposed=transposed, grad_dtype=out)
    dw = h.grad_weight(dy, x, _list(sizes, 1))
    assert _bits(h) == 0
    ref, absb = O.grouped_linear_grad_weight(_f64(dy), _f64(x), sizes)
    _close(dw.mT if transposed else dw, ref, absb, max(sizes), "dw")


# few tiles and many rows: the rows in shares, of which the last end in odd numbers or are empty
LONG = [([16384], 0, 136, 200), ([2100, 0, 3333], 40, 96, 136), ([4099, 3000], 0, 520, 264), ([0, 0, 20001], 0, 40, 72),
        ([1027], 500, 256, 256), ([3, 6200], 1, 8, 8)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("sizes,rest,N,K", LONG, ids=[f"E{len(s)}_M{sum(s) + r}_N{n}_K{k}" for s, r, n, k in LONG])
def test_weights_gradient_of_few_tiles(sizes, rest, N, K, transposed, out):
    E, M = len(sizes), sum(sizes) + rest
    x, dy, w = _randn(1, M, K), _randn(2, M, N), _randn(3, E, N, K)
    if rest:
        x[-rest:] = float("nan")
        dy[-rest:] = float("inf")
    h, g = B.GroupedLinear(w.mT.contiguous() if transposed else w, transposed=transposed, grad_dtype=out), _list(sizes, 1)
    dw = h.grad_weight(dy, x, g)
    assert _bits(h) == 0
    ref, absb = O.grouped_linear_grad_weight(_f64(dy)[:M - rest], _f64(x)[:M - rest], sizes)
    _close(dw.mT if transposed else dw, ref, absb, max(sizes), "dw")
    graph, again = torch.cuda.CUDAGraph(), torch.empty_like(dw)
    with torch.cuda.graph(graph):
        h.grad_weight(dy, x, g, out=again)
    small = h.grad_weight(dy[:64], x[:64], _list([64] + [0] * (E - 1), 1))  # one share, in the same workspace
    graph.replay()
    assert torch.equal(again, dw)
    ref, absb = O.grouped_linear_grad_weight(_f64(dy[:64]), _f64(x[:64]), [64] + [0] * (E - 1))
    _close(small.mT if transposed else small, ref, absb, 64, "dw of 64 rows")
    if out == torch.float32:
        base = torch.randn(dw.shape, generator=torch.Generator().manual_seed(5)).cuda()
        acc = base.clone()
        h.grad_weight(dy, x, g, out=acc, accumulate=True)
        assert torch.equal(acc, base + dw)  # one addition of the same sum


def _handle(E=5, N=136, K=200, seed=7, **kw):
    return B.GroupedLinear(_randn(seed, E, N, K, scale=K ** -0.5), **kw)


SOME = [70, 0, 33, 1, 150]


def test_rows_of_no_expert_stay_as_they_are_in_a_given_output():
    h, M = _handle(), sum(SOME) + 9
    x, g = _randn(1, M, 200), _list(SOME, 1)
    out = torch.full((M, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    assert h(x, g, out=out) is out
    want = h(x, g)
    assert torch.equal(out[:-9], want[:-9]) and (out[-9:] == 3).all() and not want[-9:].any()


def test_strided_rows():
    h, M = _handle(), sum(SOME)
    g = _list(SOME, 1)
    x, dy = _randn(1, M, 200), _randn(2, M, 136)
    wide_x, wide_dy = _randn(3, M, 264), _randn(4, M, 152)
    wide_x[:, 8:208], wide_dy[:, 8:144] = x, dy
    xs, dys = wide_x[:, 8:208], wide_dy[:, 8:144]
    assert torch.equal(h(xs, g), h(x, g))
    assert torch.equal(h.grad_input(dys, g), h.grad_input(dy, g))
    assert torch.equal(h.grad_weight(dys, xs, g), h.grad_weight(dy, x, g))
    for width, at in ((137, 1), (138, 2), (144, 8)):  # rows of y at any element
        wide = torch.full((M, width), 5.0, dtype=torch.bfloat16, device="cuda")
        h(x, g, out=wide[:, at:at + 136])
        assert torch.equal(wide[:, at:at + 136], h(x, g)) and (wide[:, :at] == 5).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_reaches_its_own_rows_and_expert(bad):
    """Experts' rows lie side by side in a tile: one expert's infinities and NaN must not reach the next one's sums."""
    sizes, rest = [70, 33, 1, 0, 150], 6
    M, N, K = sum(sizes) + rest, 136, 200
    x, dy, w = _randn(1, M, K), _randn(2, M, N), _randn(3, 5, N, K, scale=K ** -0.5)
    h, g = B.GroupedLinear(w, grad_dtype=torch.float32), _list(sizes, 1)
    y, dx, dw = h(x, g), h.grad_input(dy, g), h.grad_weight(dy, x, g)
    hurt_x, hurt_dy = x.clone(), dy.clone()
    for r in (70, 102, M - 1):  # expert 1's first and last row, and a row of no expert
        hurt_x[r], hurt_dy[r] = bad, bad
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[70, 102]] = False
    y2, dx2, dw2 = h(hurt_x, g), h.grad_input(hurt_dy, g), h.grad_weight(hurt_dy, hurt_x, g)
    assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
    assert not y2[~keep].isfinite().any() and not dx2[~keep].isfinite().any()
    others = [0, 2, 3, 4]
    assert torch.equal(dw2[others], dw[others]) and not dw2[1].isfinite().any()
    w2 = w.clone()
    w2[1, 5, 7] = bad
    h2 = B.GroupedLinear(w2)
    y3 = h2(x, g)
    mine = torch.zeros(M, dtype=torch.bool, device="cuda")
    mine[70:103] = True
    assert torch.equal(y3[~mine], y[~mine]) and not y3[mine][:, 5].isfinite().any()
    assert torch.equal(y3[mine][:, [0, 4, 6]], y[mine][:, [0, 4, 6]])


def test_accumulation():
    sizes = [70, 0, 33, 1, 150]
    M, N, K = sum(sizes), 136, 200
    x, dy = _randn(1, M, K), _randn(2, M, N)
    h, g = _handle(grad_dtype=torch.float32), _list(sizes, 1)
    once = h.grad_weight(dy, x, g)
    base = torch.randn(once.shape, generator=torch.Generator().manual_seed(5)).cuda()
    acc = base.clone()
    assert h.grad_weight(dy, x, g, out=acc, accumulate=True) is acc
    assert torch.equal(acc, base + once)  # one addition of the same sum
    assert torch.equal(acc[1], base[1])
    h.grad_weight(dy[:0], x[:0], torch.zeros(5, dtype=torch.int64, device="cuda"), out=acc, accumulate=True)
    assert torch.equal(acc, base + once)


def test_no_rows_at_all():
    h = _handle()
    x, dy, g = _randn(1, 0, 200), _randn(2, 0, 136), torch.zeros(5, dtype=torch.int64, device="cuda")
    assert h(x, g).shape == (0, 136) and h.grad_input(dy, g).shape == (0, 200)
    assert not h.grad_weight(dy, x, g).any()
    x, dy = _randn(1, 40, 200), _randn(2, 40, 136)  # rows, but of no expert
    assert not h(x, g).any() and not h.grad_input(dy, g).any() and not h.grad_weight(dy, x, g).any()


@pytest.mark.parametrize("kind,values,ends", [
    (1, [10, -3, 20, 5, 0], [10, 10, 30, 35, 35]),
    (1, [10, 100, 20, 5, 0], [10, 50, 50, 50, 50]),
    (1, [1 << 62, 1 << 62, 0, 0, 0], [50, 50, 50, 50, 50]),
    (0, [10, 5, 30, 40, 40], [10, 10, 30, 40, 40]),
    (0, [-1, 5, 30, 99, 50], [0, 5, 30, 50, 50]),
])
def test_a_list_that_does_not_fit_is_clamped_and_reported(kind, values, ends):
    M = 50
    x, dy = _randn(1, M, 200), _randn(2, M, 136)
    h, clean = _handle(group_list_type=kind), _handle(group_list_type=0)
    g, good = torch.tensor(values, device="cuda"), torch.tensor(ends, device="cuda")
    for call in (lambda h, g: h(x, g), lambda h, g: h.grad_input(dy, g), lambda h, g: h.grad_weight(dy, x, g)):
        got = call(h, g)
        assert _bits(h) == B.DEV_BAD_GROUP_LIST
        assert torch.equal(got, call(clean, good)) and _bits(clean) == 0


def test_other_streams_and_captured_graphs():
    h, g = _handle(), _list(SOME, 1)
    M = sum(SOME)
    x, dy = _randn(1, M, 200), _randn(2, M, 136)
    want = h(x, g), h.grad_input(dy, g), h.grad_weight(dy, x, g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = h(x, g, stream=s), h.grad_input(dy, g, stream=s), h.grad_weight(dy, x, g, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = h(x, g), h.grad_input(dy, g), h.grad_weight(dy, x, g)
    # other sizes, rows and weights in the same memory: the graph reads what is there when it runs
    g.copy_(_list([1, 200, 0, 50, 3], 1))
    x.copy_(_randn(11, M, 200)), dy.copy_(_randn(12, M, 136)), h._keep[0].copy_(_randn(13, 5, 136, 200))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, (h(x, g), h.grad_input(dy, g), h.grad_weight(dy, x, g))):
        assert torch.equal(a, b)


def test_results_do_not_change_from_call_to_call():
    sizes = torch.randint(0, 400, (24,), generator=torch.Generator().manual_seed(3)).tolist()
    M = sum(sizes)
    x, dy, w = _randn(1, M, 1032), _randn(2, M, 776), _randn(3, 24, 776, 1032)
    h, g = B.GroupedLinear(w, grad_dtype=torch.float32), _list(sizes, 1)
    first = h(x, g), h.grad_input(dy, g), h.grad_weight(dy, x, g)
    for _ in range(5):
        for a, b in zip(first, (h(x, g), h.grad_input(dy, g), h.grad_weight(dy, x, g))):
            assert torch.equal(a, b)


def test_long_sums_keep_their_bits():
    """FP32 sums of 7168 weights and of 20000 rows, all of one sign, where truncation adds up.  1024 products are 64
    additions of 16; addition i takes at most 2^-23 off a running sum that is i/64 of the whole: (1 + ... + 64) / 64 * 2^-23
    = 32.5 * 2^-23 = 3.9e-6, whatever the length.  (In one accumulator 7168 products could lose 224.5 * 2^-23 = 2.7e-5, and
    lose half of that.)  The additions to nearest of 20 such sums leave 2^-24 * 20 / 2 = 6e-7."""
    M, N, K = 20000, 64, 7168
    x, dy, w = _randn(1, M, K).abs(), _randn(2, M, N).abs(), _randn(3, 1, N, K).abs()
    h, g = B.GroupedLinear(w, out_dtype=torch.float32, grad_dtype=torch.float32), _list([M], 1)
    y, dw = h(x, g), h.grad_weight(dy, x, g)
    for got, ref in ((y, x.double() @ w[0].double().T), (dw[0], dy.double().T @ x.double())):
        assert float((got.double() - ref).norm() / ref.norm()) < 32.5 * 2 ** -23 + 6e-7


def test_experts_of_a_block_forwards_and_backwards():
    """Gate, routing step, both grouped products with SiLU between them, and the gradients of all of it, against the
    formula in 64 bits and against differences."""
    T, H, I, E, k = 96, 128, 64, 8, 2
    x, wg = _randn(1, T, H), _randn(2, E, H, scale=0.3)
    w1, w2 = _randn(3, E, H, I, scale=H ** -0.5), _randn(4, E, H, I, scale=I ** -0.5)  # [E, K, N] and [E, N, K]
    ids, weights = B.MoeGate(wg, topk=k)(x)
    routed, _ = B.route(ids, weights, x.view(torch.uint8), torch.empty((T, 2 * H // 64, 2), dtype=torch.uint8, device="cuda"), E)
    rows, g = routed["x1"].view(torch.bfloat16), routed["group_list"]
    up = B.GroupedLinear(w1, transposed=True, out_dtype=torch.float32, grad_dtype=torch.float32)
    down = B.GroupedLinear(w2, out_dtype=torch.float32, grad_dtype=torch.float32)
    z = up(rows, g)
    s = torch.sigmoid(z)
    a = (z * s).to(torch.bfloat16)
    y = down(a, g)
    dy = _randn(5, T * k, H)
    da = down.grad_input(dy, g)
    dw2 = down.grad_weight(dy, a, g)
    dz = (da.float() * (s + z * s * (1 - s))).to(torch.bfloat16)
    dx, dw1 = up.grad_input(dz, g), up.grad_weight(dz, rows, g)
    # the same in 64 bits
    sizes = g.tolist()
    expert = torch.repeat_interleave(torch.arange(E), torch.tensor(sizes)).cuda()

    def f(r, v1, v2):
        h = torch.einsum("tk,tkn->tn", r, v1[expert])
        return torch.einsum("tn,tkn->tk", h * torch.sigmoid(h), v2[expert])

    r64, a64, b64 = (t.double().requires_grad_() for t in (rows, w1, w2))
    ref = f(r64, a64, b64)
    ref.backward(dy.double())
    for name, got, want, eps in (("y", y, ref.detach(), 2 ** -8), ("dx", dx, r64.grad, 2 ** -6), ("dw1", dw1, a64.grad, 2 ** -6),
                                 ("dw2", dw2, b64.grad, 2 ** -7)):
        # roundings to BF16 on the way (a; da and dz), 2^-9 each of terms that add up at random
        far = float((got.double() - want).norm() / want.norm())
        assert far < eps, (name, far)
    # along a direction of each input: (f(p + h d) - f(p - h d)) / 2h, whose own error is of order h^2
    for i, got in enumerate((dx, dw1, dw2)):
        p = [t.detach().clone() for t in (r64, a64, b64)]
        d = torch.randn(p[i].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(9)).cuda()
        d = d / d.norm()
        h = 1e-4
        plus, minus = ([q + (sgn * h * d if j == i else 0) for j, q in enumerate(p)] for sgn in (1, -1))
        slope = ((f(*plus) - f(*minus)) / (2 * h) * dy.double()).sum()
        # |error| <= |got - grad| |d|, and |d| = 1
        assert abs(float((got.double() * d).sum() - slope)) < 2 ** -6 * float(got.double().norm())


def test_offsets_past_32_bits():
    """y, the rows and the weights' gradient of more than 2^31 elements each (the ends of them are compared)."""
    M, N, K = 66000, 32784, 64
    w = _randn(1, 2, N, K, scale=K ** -0.5)
    x = _randn(2, M, K)
    h, g = B.GroupedLinear(w), _list([M - 300, 300], 1)
    y = h(x, g)
    few = B.GroupedLinear(w)(x[-300:], _list([0, 300], 1))
    assert torch.equal(y[-300:], few)
    dx = h.grad_input(y, g)
    assert torch.equal(dx[-300:], h.grad_input(few, _list([0, 300], 1)))
    del y, dx
    torch.cuda.empty_cache()
    E, N, K = 540, 2048, 2048
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[-1] = _randn(3, N, K)
    sizes = [0] * (E - 1) + [50]
    x, dy = _randn(4, 50, K), _randn(5, 50, N)
    h, g = B.GroupedLinear(w), _list(sizes, 1)
    one, g1 = B.GroupedLinear(w[-1:].clone()), _list([50], 1)
    assert torch.equal(h(x, g), one(x, g1)) and torch.equal(h.grad_input(dy, g), one.grad_input(dy, g1))
    dw = h.grad_weight(dy, x, g)
    assert torch.equal(dw[-1], one.grad_weight(dy, x, g1)[0]) and not dw[:-1].any()


def test_a_good_call_after_a_refused_one():
    h, g = _handle(), _list(SOME, 1)
    M = sum(SOME)
    x, dy = _randn(1, M, 200), _randn(2, M, 136)
    odd = _randn(3, M, 204)[:, :200]  # rows off 16-byte boundaries
    want = h(x, g), h.grad_weight(dy, x, g)
    for bad in (lambda: h(odd, g), lambda: h.grad_weight(dy, odd, g)):
        with pytest.raises(B.GmmfrError):
            bad()
        assert torch.equal(h(x, g), want[0]) and torch.equal(h.grad_weight(dy, x, g), want[1])
