"""The few-token layer with infinite and NaN expert weights: a token's result is the formula's over the experts that it
chose, whatever the weights of those that it did not.

Tolerance where the result is finite, as in the parity tests: 2^-8 of the result and of the terms' absolute sum.
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


def _f64(t):
    return t.detach().cpu().double().numpy()


def _mx_values(codes, scale):
    v = O.mx_values(codes.numpy(), scale.numpy())
    k = np.arange(codes.shape[1])
    s = scale.numpy()[:, k // 64, :, (k // 32) % 2].transpose(1, 0, 2)
    return np.where((codes.numpy() & 127 == 127) | (s == 255), np.nan, v)


# column tiles that one CTA has to itself (few tiles in all), and tiles cut between CTAs; odd sizes; 64 tokens
SIZES = [dict(T=2, H=1024, E=4, I=64, shared_I=0, topk=1), dict(T=6, H=256, E=16, I=64, shared_I=64, topk=4),
         dict(T=13, H=1032, E=24, I=200, shared_I=72, topk=3), dict(T=64, H=512, E=40, I=136, shared_I=0, topk=6)]


@pytest.mark.parametrize("where,mx", [(w, m) for w in ("down", "down column", "up", "scale") for m in (False, True) if m or w != "scale"],
                         ids=lambda v: {False: "bf16", True: "mxfp8"}.get(v, v))
@pytest.mark.parametrize("c", SIZES, ids=lambda c: f"T{c['T']}-H{c['H']}-E{c['E']}-I{c['I']}-s{c['shared_I']}-k{c['topk']}")
def test_weights_that_a_token_did_not_choose(c, where, mx):
    T, H, E, I, sI, topk = (c[k] for k in ("T", "H", "E", "I", "shared_I", "topk"))
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    wg = (torch.randn((E, H), generator=g) * H ** -0.5).to(torch.bfloat16)
    residual = torch.randn((T, H), generator=g).to(torch.bfloat16)
    w, s = {}, {}
    for name, n, K, N in (("w13", E, H, 2 * I), ("w2", E, I, H), ("shared_w13", 1, H, 2 * sI), ("shared_w2", 1, sI, H)):
        if K == 0 or N == 0:
            continue
        v = torch.randn((n, K, N), generator=g)
        if mx:
            w[name] = v.to(torch.float8_e4m3fn).view(torch.uint8)
            s[name] = torch.randint(120, 126, (n, -(-K // 64), N, 2), generator=g).to(torch.uint8)
        else:
            w[name] = (v * K ** -0.5).to(torch.bfloat16)
    # the experts that the fewest tokens chose get bad weights, as many as leave half of the tokens without one
    ids = B.MoeGate(wg.cuda(), topk=topk)(x.cuda())[0].cpu()
    bad = []
    for e in sorted(ids.unique().tolist(), key=lambda e: (int((ids == e).sum()), e)):
        if 2 * int(torch.isin(ids, torch.tensor(bad + [e])).any(1).sum()) <= T:
            bad.append(e)
    assert bad
    nan = 127 if mx else float("nan")
    inf = 255 if mx else float("-inf")  # E4M3 has no infinity
    for e in bad:
        if where == "down":
            w["w2"][e, I // 3, :] = inf
            w["w2"][e, I - 1, ::2] = nan
        elif where == "down column":
            w["w2"][e, :, H - 3] = nan
        elif where == "up":
            w["w13"][e, H // 2, I + 5] = nan
            w["w13"][e, 3, 2] = inf
        else:
            s["w2"][e, 0, 7, 0] = 255
    dev = {k: v.cuda() for k, v in w.items()}
    sc = {k + "_scale": v.cuda() for k, v in s.items()}
    shared = {k: dev[k][0] for k in dev if k.startswith("shared")}
    shared.update({k: sc[k][0] for k in sc if k.startswith("shared")})
    layer = B.MoeLayer(wg.cuda(), dev["w13"], dev["w2"], w13_scale=sc.get("w13_scale"), w2_scale=sc.get("w2_scale"), **shared, topk=topk)
    chosen = torch.empty((T, topk), dtype=torch.int32, device="cuda")
    wt = torch.empty((T, topk), device="cuda")
    out = layer(x.cuda(), residual=residual.cuda(), topk_ids=chosen, topk_weights=wt)
    values = {k: _mx_values(w[k], s[k]) if mx else _f64(w[k]) for k in w}
    with np.errstate(all="ignore"):
        ref, absb = O.moe_layer(_f64(x), chosen.cpu().numpy(), _f64(wt), values["w13"], values["w2"],
                                *((values["shared_w13"][0], values["shared_w2"][0]) if sI else (None, None)), residual=_f64(residual))
        got = _f64(out)
        fine = np.isfinite(ref)
        clean = ~np.isin(chosen.cpu().numpy(), bad).any(1)
        assert clean.any() and fine[clean].all()
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
        assert np.all((np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + absb) + 1e-30)[fine])
    assert torch.equal(out.view(torch.int16), layer(x.cuda(), residual=residual.cuda()).view(torch.int16))


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,H,E,I,topk", [(3, 1024, 4, 64, 1), (40, 520, 16, 136, 4)])
def test_tokens_and_weights_at_once(T, H, E, I, topk, value, mx):
    """A token that is not finite itself, beside an expert of NaN weights that some of the others chose."""
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    wg = (torch.randn((E, H), generator=g) * H ** -0.5).to(torch.bfloat16)
    x[1] = value
    w13, w2 = torch.randn((E, H, 2 * I), generator=g), torch.randn((E, I, H), generator=g)
    scales = {}
    if mx:
        w13, w2 = (w.to(torch.float8_e4m3fn) for w in (w13, w2))
        scales = {n + "_scale": torch.full((E, -(-k // 64), c, 2), 122, dtype=torch.uint8).cuda() for n, k, c in (("w13", H, 2 * I), ("w2", I, H))}
    else:
        w13, w2 = (w * H ** -0.5 for w in (w13, w2))
    bad = int(B.MoeGate(wg.cuda(), topk=topk)(x.cuda())[0][0, 0])
    clean = [w.to(w.dtype if mx else torch.bfloat16).cuda() for w in (w13, w2)]
    spoilt = clean[1].clone()
    spoilt.view(torch.uint8 if mx else torch.int16)[bad] = 0x7F if mx else 0x7FC0
    chosen = torch.empty((T, topk), dtype=torch.int32, device="cuda")
    ref = B.MoeLayer(wg.cuda(), *clean, **scales, topk=topk)(x.cuda())
    out = B.MoeLayer(wg.cuda(), clean[0], spoilt, **scales, topk=topk)(x.cuda(), topk_ids=chosen, topk_weights=torch.empty((T, topk), device="cuda"))
    got, want, has = _f64(out), _f64(ref), (chosen == bad).any(1).cpu().numpy()
    assert np.isnan(got[1]).all() and np.isnan(got[has]).all() and not has.all()
    for t in range(T):
        if t != 1 and not has[t]:
            # the same terms, added in another order
            assert np.all(np.abs(got[t] - want[t]) <= 2.0 ** -7 * np.abs(want[t]) + 2.0 ** -8 * np.abs(want[t]).max())
