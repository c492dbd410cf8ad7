"""GPU parity of the router, the few-token MoE layer and the dense product against float64 oracles.

Tolerances, from the arithmetic:
  sums      FP32 additions of exact BF16 products.  A tensor core adds 16 products at a time to the running
            sum and may truncate: K/16 additions of at most 2^-23 relative each; K/8 * 2^-23 * sum |x w| leaves a
            factor of two and is still below one lost term (sum |x w| / K) for K < 8192.
  BF16      one rounding of the result is 2^-9 relative; results computed apart may round to neighbours: 2^-8.
  layer     besides, the SwiGLU value is rounded to 8 bits before the down product: 2^-9 of every term, taken
            as 2^-8 * sum |terms| with what the sums before it leave.
  softmax   exponentials and sums of E values in FP32: 2^-18 relative is 64 ulp.
"""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_mxfp8_gb300 import binding as B
from moe_grouped_gemm_mxfp8_gb300 import build as build_mod
from oracle import moe as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.load()


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def _f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------------------------------- router
def _check_gate(x, w, logits_exact=None, **rule):
    """The logits against the exact product, then the choice against the oracle's on those logits."""
    T, E = x.shape[0], w.shape[0]
    bias = rule.get("select_bias")
    dev = {**rule, "select_bias": None if bias is None else bias.cuda()}
    gate = B.MoeGate(w.cuda(), **dev)
    logits = torch.full((T, E), 7.0, device="cuda")
    xd = x if x.is_cuda else x.cuda()
    ids, wt = gate(xd, logits=logits)
    ids2, wt2 = gate(xd)  # without the logits: the same choice
    assert torch.equal(ids, ids2) and torch.equal(wt.view(torch.int32), wt2.view(torch.int32))
    got = _f64(logits)
    xf, wf = _f64(x), _f64(w)
    if logits_exact is None:
        err = np.abs(got - xf @ wf.T)
        tol = x.shape[1] / 8 * 2.0 ** -23 * (np.abs(xf) @ np.abs(wf).T)
        assert np.all(err <= tol), (err / np.maximum(tol, 1e-300)).max()
    ids, wt = ids.cpu().numpy().astype(np.int64), _f64(wt)
    r = {**rule, "select_bias": None if bias is None else _f64(bias)}
    ref_ids, _, s = O.gate_select(got, **r)
    assert all(len(set(row)) == len(row) for row in ids.tolist()) and ids.min(initial=0) >= 0 and ids.max(initial=0) < E
    # a choice may differ from the oracle's only between scores that FP32 cannot tell apart
    a, b = np.take_along_axis(s, ids, 1), np.take_along_axis(s, ref_ids, 1)
    with np.errstate(invalid="ignore"):
        same = (ids == ref_ids) | (np.abs(a - b) <= 2.0 ** -18 * (np.abs(b) + 1e-30))
    assert same.all()
    p = O.gate_probabilities(got, rule.get("scoring", "softmax"))
    ref = np.take_along_axis(p, ids, 1)
    if rule.get("renormalise", True):
        ref = ref / (ref.sum(-1, keepdims=True) + 1e-20)
    ref = ref * rule.get("scale", 1.0)
    assert np.all(np.abs(wt - ref) <= 2.0 ** -18 * np.abs(ref) + 1e-37)
    return ids, wt


GATES = [
    dict(T=1, H=2048, E=256, topk=8, scoring="sigmoid", bias=True, n_group=8, topk_group=4, scale=2.5),
    dict(T=1, H=8, E=1, topk=1, scoring="softmax"),
    dict(T=3, H=72, E=7, topk=7, scoring="softmax", renormalise=False),
    dict(T=65, H=264, E=33, topk=5, scoring="sigmoid", n_group=11, topk_group=3, group_top=1),
    dict(T=129, H=520, E=160, topk=6, scoring="softmax"),
    dict(T=200, H=128, E=64, topk=32, scoring="sigmoid", bias=True, n_group=64, topk_group=40, group_top=1),
    dict(T=257, H=136, E=512, topk=8, scoring="softmax", n_group=4, topk_group=1),
    dict(T=70, H=64, E=1024, topk=8, scoring="sigmoid", bias=True),
    dict(T=1000, H=2048, E=256, topk=8, scoring="sigmoid", bias=True, n_group=8, topk_group=4, scale=2.5),
    dict(T=2500, H=1288, E=200, topk=3, scoring="softmax"),
    dict(T=4100, H=256, E=48, topk=2, scoring="softmax"),
    dict(T=1700, H=264, E=512, topk=8, scoring="softmax", n_group=4, topk_group=1),
    dict(T=1900, H=200, E=300, topk=8, scoring="sigmoid", bias=True, n_group=50, topk_group=9),
    dict(T=961, H=72, E=7, topk=7, scoring="softmax", renormalise=False),
    dict(T=961, H=128, E=64, topk=32, scoring="sigmoid", n_group=64, topk_group=33, group_top=1),
    dict(T=40000, H=64, E=36, topk=5, scoring="sigmoid", n_group=12, topk_group=5),
    dict(T=530, H=64, E=600, topk=8, scoring="softmax"),
    dict(T=1025, H=72, E=7, topk=7, scoring="softmax", renormalise=False),
    dict(T=1025, H=128, E=64, topk=32, scoring="sigmoid", n_group=64, topk_group=33, group_top=1),
    dict(T=300, H=200, E=500, topk=32, scoring="sigmoid", n_group=5, topk_group=2),
    dict(T=530, H=136, E=129, topk=20, scoring="softmax"),
    dict(T=9, H=2048, E=16, topk=4, scoring="softmax"),
    dict(T=5, H=72, E=600, topk=20, scoring="sigmoid", bias=True),
    dict(T=270, H=64, E=600, topk=32, scoring="sigmoid", bias=True, n_group=30, topk_group=7),
    dict(T=600, H=64, E=1000, topk=17, scoring="softmax", bias=True),
]


@pytest.mark.parametrize("c", GATES, ids=lambda c: f"T{c['T']}-H{c['H']}-E{c['E']}-k{c['topk']}-{c['scoring']}-g{c.get('n_group', 1)}")
def test_gate_parity(c):
    c = dict(c)
    T, H, E = c.pop("T"), c.pop("H"), c.pop("E")
    g = _gen(T + H + E)
    x, w = _randn(g, T, H), _randn(g, E, H, scale=1.3 / H ** 0.5)
    if c.pop("bias", False):
        c["select_bias"] = _randn(g, E, scale=0.05, dtype=torch.float32)
    _check_gate(x, w, **c)


@pytest.mark.parametrize("T", [1, 5, 300, 1111])
def test_gate_ties_go_to_the_lowest_index(T):
    # one-hot rows pick small whole numbers out of the weights: logits are exact, ties are ties
    g = _gen(T)
    E, H = 96, 64
    w = torch.randint(-2, 3, (E, H), generator=g).to(torch.bfloat16)
    x = torch.zeros(T, H)
    x[torch.arange(T), torch.randint(0, H, (T,), generator=g)] = 1
    for rule in (dict(topk=8, scoring="softmax"), dict(topk=8, scoring="sigmoid", n_group=8, topk_group=3),
                 dict(topk=8, scoring="sigmoid", n_group=12, topk_group=2, group_top=1)):
        ids, _ = _check_gate(x.to(torch.bfloat16), w, logits_exact=True, **rule)
        logits = _f64(x) @ _f64(w).T
        want, _, _ = O.gate_select(logits, **rule)
        assert np.array_equal(ids, want)


@pytest.mark.parametrize("T", [2, 200, 1777])
def test_gate_masked_and_infinite_scores(T):
    g = _gen(7)
    E, H = 64, 64
    x, w = _randn(g, T, H), _randn(g, E, H, scale=0.2)
    # all but four experts masked out of the selection, by -inf and by the type's lowest value
    for low in (-float("inf"), torch.finfo(torch.float32).min):
        bias = torch.full((E,), low)
        bias[[3, 17, 40, 63]] = 0.0
        for groups in (dict(), dict(n_group=8, topk_group=3)):
            gate = B.MoeGate(w.cuda(), topk=8, scoring="sigmoid", select_bias=bias.cuda(), **groups)
            ids, wt = gate(x.cuda())
            ids = ids.cpu().numpy()
            if not groups:
                assert all(set(r[:4]) == {3, 17, 40, 63} for r in ids.tolist())
                assert all(r[4:] == [0, 1, 2, 4] for r in ids.tolist())  # the rest are equal: lowest indices
            assert torch.isfinite(wt).all()
    # a mask that leaves nothing: every score equal, the lowest indices
    ids, _ = B.MoeGate(w.cuda(), topk=5, scoring="sigmoid", select_bias=torch.full((E,), -float("inf"), device="cuda"))(x.cuda())
    assert all(r == [0, 1, 2, 3, 4] for r in ids.tolist())
    # logits that are all -inf: nothing to weigh
    xi = torch.full((T, H), -float("inf"), dtype=torch.bfloat16)
    wi = torch.zeros(E, H, dtype=torch.bfloat16)
    wi[:, 0] = 1.0
    xi[:, 1:] = 0.0
    ids, wt = B.MoeGate(wi.cuda(), topk=4)(xi.cuda())
    assert all(r == [0, 1, 2, 3] for r in ids.tolist()) and (wt == 0).all()
    # NaN in one token: its weights are NaN, the other tokens do not notice
    xn = x.clone()
    xn[1] = float("nan")
    ids, wt = B.MoeGate(w.cuda(), topk=4)(xn.cuda())
    ref_ids, ref_wt = B.MoeGate(w.cuda(), topk=4)(x.cuda())
    keep = [t for t in range(T) if t != 1]
    assert ids[1].tolist() == [0, 1, 2, 3] and torch.isnan(wt[1]).all()
    assert torch.equal(ids[keep], ref_ids[keep]) and torch.equal(wt[keep], ref_wt[keep])


@pytest.mark.parametrize("T", [3, 333, 1777])
def test_gate_strided_rows_int64_ids_and_another_stream(T):
    g = _gen(11)
    wide = _randn(g, T, 200).cuda()
    w = _randn(g, 40, 128, scale=0.1)
    x = wide[:, 16:144]
    ref = B.MoeGate(w.cuda(), topk=3)(x.contiguous())
    ids, wt = B.MoeGate(w.cuda(), topk=3, ids_dtype=torch.int64)(x)
    assert ids.dtype == torch.int64 and torch.equal(ids, ref[0].long()) and torch.equal(wt, ref[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gate = B.MoeGate(w.cuda(), topk=3)
    torch.cuda.synchronize()
    ids, wt = gate(x, stream=s)
    s.synchronize()
    assert torch.equal(ids, ref[0]) and torch.equal(wt, ref[1])
    assert B.MoeGate(w.cuda(), topk=3)(x[:0])[0].shape == (0, 3)


def test_gate_feeds_the_routing_step():
    g = _gen(3)
    T, H, E = 50, 128, 16
    x, w = _randn(g, T, H), _randn(g, E, H, scale=0.1)
    ids, wt = B.MoeGate(w.cuda(), topk=4, ids_dtype=torch.int64)(x.cuda())
    codes = torch.randint(0, 255, (T, H), generator=g, dtype=torch.int32).to(torch.uint8).cuda()
    scale = torch.full((T, 2, 2), 127, dtype=torch.uint8, device="cuda")
    o, ws = B.route(ids, wt, codes, scale, E)
    assert B.gmmfr_check_device_errors(ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert int(o["group_list"].sum()) == T * 4
    order = np.argsort(ids.cpu().numpy().reshape(-1), kind="stable")
    assert np.array_equal(o["perm"].cpu().numpy(), order)
    assert torch.equal(o["logit"], wt.reshape(-1)[o["perm"].long()])


# ------------------------------------------------------------------------------------------- layer
def _layer_inputs(g, T, H, E, I, shared_I, mx, scale=1.0):
    d = dict(x=_randn(g, T, H), wg=_randn(g, E, H, scale=1.3 / H ** 0.5))
    for pre, n, i in (("", E, I), ("shared_", 1, shared_I)):
        if i == 0:
            continue
        if mx:
            for name, K, N in (("w13", H, 2 * i), ("w2", i, H)):
                d[pre + name] = (torch.randn((n, K, N), generator=g)).to(torch.float8_e4m3fn)
                e = 127 - round(np.log2(K) / 2)
                d[pre + name.replace("w", "s")] = torch.randint(e - 3, e + 3, (n, -(-K // 64), N, 2), generator=g).to(torch.uint8)
        else:
            d[pre + "w13"] = _randn(g, n, H, 2 * i, scale=scale * H ** -0.5)
            d[pre + "w2"] = _randn(g, n, i, H, scale=scale * i ** -0.5)
    return d


def _values(d, name):
    if d[name].dtype == torch.bfloat16:
        return _f64(d[name])
    return O.mx_values(d[name].view(torch.uint8).numpy(), d[name.replace("w", "s", 1) if not name.startswith("shared_")
                                                             else "shared_s" + name[len("shared_w"):]].numpy())


def _make_layer(d, **rule):
    c = {k: v.cuda() for k, v in d.items()}
    sh = {}
    if "shared_w13" in c:
        sh = dict(shared_w13=c["shared_w13"][0], shared_w2=c["shared_w2"][0])
        if "shared_s13" in c:
            sh.update(shared_w13_scale=c["shared_s13"][0], shared_w2_scale=c["shared_s2"][0])
    return B.MoeLayer(c["wg"], c["w13"], c["w2"], w13_scale=c.get("s13"), w2_scale=c.get("s2"), **sh, **rule)


def _check_layer(d, layer, topk, residual=None, x=None):
    x = d["x"].cuda() if x is None else x
    T = x.shape[0]
    ids = torch.full((T, topk), -1, dtype=torch.int32, device="cuda")
    wt = torch.zeros((T, topk), device="cuda")
    out = layer(x, residual=residual, topk_ids=ids, topk_weights=wt)
    again = layer(x, residual=residual)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # deterministic, and without the choice
    sh = (_values(d, "shared_w13")[0], _values(d, "shared_w2")[0]) if "shared_w13" in d else (None, None)
    ref, absb = O.moe_layer(_f64(x), ids.cpu().numpy(), _f64(wt), _values(d, "w13"), _values(d, "w2"), *sh,
                            residual=None if residual is None else _f64(residual))
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * absb + 1e-30
    err = np.abs(_f64(out) - ref)
    assert np.all(err <= tol), (err / tol).max()
    return out, ids, wt


LAYERS = [
    dict(T=1, H=256, E=16, I=64, shared_I=64, topk=4),
    dict(T=1, H=72, E=4, I=8, shared_I=0, topk=1),
    dict(T=2, H=2048, E=32, I=512, shared_I=512, topk=8, scoring="sigmoid", n_group=8, topk_group=4, scale=2.5),
    dict(T=5, H=200, E=9, I=136, shared_I=72, topk=3),
    dict(T=16, H=512, E=24, I=192, shared_I=384, topk=6),
    dict(T=17, H=264, E=40, I=72, shared_I=0, topk=2),
    dict(T=33, H=1032, E=8, I=264, shared_I=264, topk=8),
    dict(T=64, H=384, E=64, I=128, shared_I=128, topk=8, scoring="sigmoid"),
    dict(T=64, H=128, E=300, I=64, shared_I=0, topk=32),
    dict(T=63, H=640, E=3, I=328, shared_I=8, topk=1),
]


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("c", LAYERS, ids=lambda c: f"T{c['T']}-H{c['H']}-E{c['E']}-I{c['I']}-s{c['shared_I']}-k{c['topk']}")
def test_layer_parity(c, mx):
    c = dict(c)
    T, H, E, I, sI = (c.pop(k) for k in ("T", "H", "E", "I", "shared_I"))
    g = _gen(T + H + E + I)
    d = _layer_inputs(g, T, H, E, I, sI, mx)
    layer = _make_layer(d, **c)
    residual = _randn(g, T, H).cuda() if T % 2 else None
    out, ids, wt = _check_layer(d, layer, c["topk"], residual)
    gate = B.MoeGate(d["wg"].cuda(), **c)  # the layer's choice is the gate's (FP32 sums may differ in order)
    gi, gw = gate(d["x"].cuda())
    assert (gi == ids).float().mean() > 0.98 and torch.allclose(gw.sort(-1).values, wt.sort(-1).values, rtol=1e-3, atol=1e-6)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
def test_layer_all_tokens_on_the_same_experts(mx):
    g = _gen(5)
    d = _layer_inputs(g, 64, 256, 32, 128, 64, mx)
    bias = torch.zeros(32)
    bias[[1, 30]] = 10.0  # a selection bias that sends every token to two experts
    layer = _make_layer(d, topk=2, scoring="sigmoid", select_bias=bias.cuda())
    _, ids, _ = _check_layer(d, layer, 2)
    assert {frozenset(r) for r in ids.tolist()} == {frozenset((1, 30))}


def test_layer_sizes_in_turn_strides_alias_and_streams():
    g = _gen(6)
    d = _layer_inputs(g, 40, 256, 16, 64, 64, False)
    layer = _make_layer(d, topk=4)
    for T in (40, 1, 17, 40, 3, 0):  # one handle, its workspace reused by smaller and larger calls
        x = d["x"][:T].cuda()
        if T:
            _check_layer(d, layer, 4, x=x)
        else:
            assert layer(x).shape == (0, 256)
    wide = torch.zeros((9, 512), dtype=torch.bfloat16, device="cuda")
    wide[:, 128:384] = d["x"][:9].cuda()
    res = _randn(g, 9, 300).cuda()
    ref = layer(d["x"][:9].cuda(), residual=res[:, :256].contiguous())
    out = torch.zeros((9, 264), dtype=torch.bfloat16, device="cuda")
    layer(wide[:, 128:384], residual=res[:, :256], out=out[:, :256])
    assert torch.equal(out[:, :256], ref) and (out[:, 256:] == 0).all()
    inplace = res[:, :256].clone()
    layer(d["x"][:9].cuda(), residual=inplace, out=inplace)
    assert torch.equal(inplace, ref)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = layer(d["x"][:9].cuda(), stream=s)
    b = layer(d["x"][:9].cuda())
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_layer_prepared_weights_serve_the_grouped_ffn_too():
    g = _gen(8)
    H, I, E, T = 256, 64, 8, 12
    d = _layer_inputs(g, T, H, E, I, 0, False)
    layer = _make_layer(d, topk=1, renormalise=True)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    out = layer(d["x"].cuda(), topk_ids=ids, topk_weights=torch.zeros((T, 1), device="cuda"))
    order = torch.argsort(ids[:, 0].long(), stable=True)
    cum = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    cum[1:] = torch.bincount(ids[:, 0].long(), minlength=E).cumsum(0).to(torch.int32)
    y, _ = B.ffn(d["x"].cuda()[order].contiguous(), layer._prepared, cum, H, I, E)
    a, b = _f64(out[order]), _f64(y)
    sw = 2.0 ** -7 * (np.abs(a).max() + 1)
    assert np.abs(a - b).max() <= sw


def test_layer_nan_and_infinite_tokens_stay_in_their_rows():
    g = _gen(9)
    d = _layer_inputs(g, 6, 256, 16, 64, 64, False)
    layer = _make_layer(d, topk=4)
    ref = layer(d["x"].cuda())
    x = d["x"].clone()
    x[2] = float("nan")
    x[4, 7] = float("inf")
    out = layer(x.cuda())
    keep = [0, 1, 3, 5]
    # the experts that the NaN row falls to may move the places where other rows' sums are split
    a, b = _f64(out[keep]), _f64(ref[keep])
    assert np.all(np.abs(a - b) <= 2.0 ** -7 * np.abs(b) + 2.0 ** -8 * np.abs(b).max())
    assert torch.isnan(out[2]).all()


# ------------------------------------------------------------------------------------------- dense product
def _check_linear(x, w, act="none", bias=None, residual=None, out_dtype=torch.bfloat16, **kw):
    xd, wd = (t if t.is_cuda else t.cuda() for t in (x, w))
    lin = B.Linear(wd, bias=None if bias is None else bias.cuda(), activation=act, out_dtype=out_dtype)
    rd = None if residual is None else (residual if residual.is_cuda else residual.cuda())
    y = lin(xd, residual=rd, **kw)
    ref, a = O.linear(_f64(x), _f64(w), None if bias is None else _f64(bias), None if residual is None else _f64(residual), act)
    tol = (2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -20) * np.abs(ref) + x.shape[1] / 8 * 2.0 ** -23 * a + 1e-30
    err = np.abs(_f64(y) - ref)
    assert np.all(err <= tol), (err / tol).max()
    assert torch.equal(y, lin(xd, residual=rd))  # deterministic
    return y


LINEARS = [(1, 1, 1), (1, 2048, 2048), (3, 5, 7), (2, 130, 264), (7, 1000, 520), (16, 256, 512), (17, 77, 1032), (33, 4096, 136),
           (48, 300, 1024), (64, 64, 64), (65, 129, 72), (100, 640, 1000), (128, 256, 128), (200, 257, 2051), (300, 1000, 520),
           (777, 517, 1288), (1025, 384, 4096), (1, 333, 7168), (5, 2000, 1023), (20, 2000, 4096), (100, 20000, 200),
           (128, 2048, 2048)]


@pytest.mark.parametrize("act", list(B.ACTIVATIONS))
@pytest.mark.parametrize("M,N,K", LINEARS, ids=lambda v: str(v))
def test_linear_parity(M, N, K, act):
    g = _gen(M * 31 + N * 7 + K)
    rows = 2 * N if act == "swiglu" else N
    x, w = _randn(g, M, K), _randn(g, rows, K, scale=K ** -0.5)
    pick = (M + N + K + len(act)) % 4
    bias = _randn(g, rows, scale=0.5) if pick & 1 else None
    residual = _randn(g, M, N) if pick & 2 else None
    _check_linear(x, w, act, bias, residual, torch.float32 if (N + len(act)) % 2 else torch.bfloat16)


@pytest.mark.parametrize("M,N,K,act,unaligned", [(777, 5120, 1288, "gelu_tanh", False), (1030, 4096, 2048, "none", False),
                                                 (777, 2560, 1288, "swiglu", False), (777, 5125, 1289, "silu", True)])
def test_linear_rows_past_the_last_full_tile(M, N, K, act, unaligned):
    """Sizes whose last rows are a launch of their own beside the others'."""
    g = _gen(M + N + K)
    rows = 2 * N if act == "swiglu" else N
    x, w = _randn(g, M, K).cuda(), _randn(g, rows, K, scale=K ** -0.5).cuda()
    bias, residual = _randn(g, rows, scale=0.5).cuda(), _randn(g, M, N + 3).cuda()[:, 1:1 + N]
    _check_linear(x, w, act, bias, residual, torch.float32 if unaligned else torch.bfloat16)
    # what follows on the stream sees all rows, and what came before is seen by all
    lin, back = B.Linear(w, bias=bias, activation=act), B.Linear(_randn(g, 64, N, scale=N ** -0.5).cuda())
    outs = []
    for wait in (True, False):
        y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
        xs = torch.zeros_like(x)
        torch.cuda.synchronize()
        for i in range(4):
            xs.copy_(x).mul_(1 + i)
            if wait:
                torch.cuda.synchronize()
            lin(xs, out=y)
            if wait:
                torch.cuda.synchronize()
            outs.append(back(y))
    for a, b in zip(outs[:4], outs[4:]):
        assert torch.equal(a, b)


def test_calls_in_a_cuda_graph():
    g = _gen(4)
    d = _layer_inputs(g, 24, 256, 16, 64, 64, False)
    layer = _make_layer(d, topk=4)
    gate = B.MoeGate(d["wg"].cuda(), topk=4)
    x = d["x"].cuda()
    calls = [lambda: layer(x, residual=x), lambda: gate(x)[1]]
    for M, N, K in ((1, 64, 72), (100, 640, 1000), (1030, 4096, 2048)):
        lin, y = B.Linear(_randn(g, N, K, scale=K ** -0.5).cuda()), _randn(g, M, K).cuda()
        calls.append(lambda lin=lin, y=y: lin(y))
    eager = [c().clone() for c in calls]  # sizes the workspaces
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for c in calls:
            c()
        with torch.cuda.graph(graph, stream=stream):
            captured = [c() for c in calls]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, captured):
        assert torch.equal(a, b)


def test_error_words_are_clean():
    g = _gen(3)
    s = torch.cuda.current_stream().cuda_stream

    def clean(handle):
        ws = handle._spaces[s][0]
        assert B.gmmfr_check_device_errors(ws, s) == 0

    for M, N, K in ((1, 64, 64), (16, 256, 512), (100, 640, 1000), (300, 1000, 520), (1030, 4096, 2048)):
        lin = B.Linear(_randn(g, N, K).cuda())
        lin(_randn(g, M, K).cuda())
        clean(lin)
    for T in (5, 1500):
        gate = B.MoeGate(_randn(g, 64, 128).cuda(), topk=4)
        gate(_randn(g, T, 128).cuda())
        clean(gate)
    d = _layer_inputs(g, 6, 256, 16, 64, 64, False)
    layer = _make_layer(d, topk=4)
    layer(d["x"].cuda())
    clean(layer)


@pytest.mark.parametrize("M", [1, 20, 150])
@pytest.mark.parametrize("off,ld", [(0, 264), (8, 272), (1, 264), (3, 271)])
def test_linear_strides_and_alignment(M, off, ld):
    g = _gen(M + off + ld)
    N, K = 100, 256
    xw, ww, rw = _randn(g, M, ld).cuda(), _randn(g, N, ld, scale=0.1).cuda(), _randn(g, M, 2 * N + 3).cuda()
    x, w, r = xw[:, off:off + K], ww[:, off:off + K], rw[:, 1:1 + N]
    ref = _check_linear(x, w, "silu", residual=r)
    buf = torch.full((M, N + 5), 3.0, dtype=torch.bfloat16, device="cuda")
    lin = B.Linear(w, activation="silu")
    lin(x, residual=r, out=buf[:, 2:2 + N])
    assert torch.equal(buf[:, 2:2 + N], ref) and (buf[:, :2] == 3).all() and (buf[:, 2 + N:] == 3).all()
    inplace = r.clone()  # of its own: one row of r is contiguous already
    lin(x, residual=inplace, out=inplace)
    assert torch.equal(inplace, ref)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = lin(x, residual=r, stream=s)
    s.synchronize()
    assert torch.equal(y, ref)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_infinities_and_nan_stay_in_their_rows_and_columns(M):
    g = _gen(M)
    N, K = 200, 264
    x, w = _randn(g, M, K), _randn(g, N, K, scale=0.1)
    ref = B.Linear(w.cuda())(x.cuda())
    w2 = w.clone()
    w2[N - 1, 5] = float("nan")
    y = B.Linear(w2.cuda())(x.cuda())
    assert torch.isnan(y[:, N - 1]).all() and torch.equal(y[:, :N - 1], ref[:, :N - 1])
    if M > 1:
        x2 = x.clone()
        x2[M - 1, K - 1] = float("inf")
        y = B.Linear(w.cuda())(x2.cuda())
        assert torch.equal(y[:M - 1], ref[:M - 1]) and not torch.isfinite(y[M - 1]).any()


def test_linear_empty():
    w = torch.zeros((6, 8), dtype=torch.bfloat16, device="cuda")
    assert B.Linear(w)(torch.zeros((0, 8), dtype=torch.bfloat16, device="cuda")).shape == (0, 6)


def test_handles_refuse_what_does_not_fit():
    w = torch.zeros((6, 8), dtype=torch.bfloat16, device="cuda")
    lin = B.Linear(w)
    x = torch.zeros((3, 8), dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x[:, :7], x.cpu(), x.t(), x[0], x[:1].expand(3, 8)):
        with pytest.raises(ValueError):
            lin(bad)
    for bad in (x[:, :6].float(), x[:2, :6], x[:, :5]):
        with pytest.raises(ValueError):
            lin(x, residual=bad)
    with pytest.raises(ValueError):
        lin(x, out=torch.zeros((3, 6), device="cuda"))
    for kw in (dict(activation="tanh"), dict(bias=torch.zeros(5, dtype=torch.bfloat16, device="cuda")), dict(out_dtype=torch.float16),
               dict(bias=torch.zeros(6, device="cuda"))):
        with pytest.raises(ValueError):
            B.Linear(w, **kw)
    with pytest.raises(ValueError):
        B.Linear(w[:5], activation="swiglu")
    gate = B.MoeGate(w, topk=2)
    with pytest.raises(ValueError):
        gate(x.float())
    with pytest.raises(ValueError):
        gate(x, ids=torch.zeros((3, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        B.MoeGate(w, topk=2, scoring="tanh")
    with pytest.raises(B.GmmfrError):
        B.MoeGate(w, topk=7)
    with pytest.raises(ValueError):
        B.MoeLayer(w, torch.zeros((6, 8, 16), dtype=torch.float16, device="cuda"),
                   torch.zeros((6, 8, 8), dtype=torch.float16, device="cuda"), topk=2)
    layer = B.MoeLayer(w, torch.zeros((6, 8, 16), dtype=torch.bfloat16, device="cuda"),
                       torch.zeros((6, 8, 8), dtype=torch.bfloat16, device="cuda"), topk=2)
    with pytest.raises(B.GmmfrError):
        layer(torch.zeros((65, 8), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        layer(x, residual=x[:, :6])
