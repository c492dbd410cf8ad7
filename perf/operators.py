"""Measured cases of the mixture-of-experts serving operators: the router (``gate``), the whole
layer for a few tokens (``layer``) and the dense product with a fused epilogue (``linear``).

Each case runs in two forms on the same inputs: ``own = False`` computes the operator with
elementary torch operations in 32 bits, rounded once at the end; ``own = True`` makes the calls a
user makes of the library.  ``exact`` gives the definition's value in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # router of one decoded token: 256 experts in 8 groups, 8 chosen (LLaDA2.0-mini's sizes)
        dict(name="gate 1", op="gate", T=1, H=2048, E=256, topk=8, scoring="sigmoid", bias=True, n_group=8,
             topk_group=4, scale=2.5),
        # a mixed batch of prompts' tails and decoded tokens, softmax scores, no groups
        dict(name="gate 333", op="gate", T=333, H=5120, E=160, topk=6, scoring="softmax", bias=False, n_group=1,
             topk_group=1, scale=1.0),
        # a long prompt chunk
        dict(name="gate 16384", op="gate", T=16384, H=2048, E=256, topk=8, scoring="sigmoid", bias=True, n_group=8,
             topk_group=4, scale=2.5),
        # one sequence decoding: nine experts' weights (eight and the shared one)
        dict(name="layer bf16 1", op="layer", T=1, H=2048, E=256, I=512, shared_I=512, topk=8, scoring="sigmoid",
             bias=True, n_group=8, topk_group=4, scale=2.5, weights="bf16", residual=True),
        # a small decoding batch: most experts have one token
        dict(name="layer bf16 13", op="layer", T=13, H=2048, E=256, I=512, shared_I=512, topk=8, scoring="sigmoid",
             bias=True, n_group=8, topk_group=4, scale=2.5, weights="bf16", residual=True),
        # the largest decoding batch of the form: nearly every expert's weights are read
        dict(name="layer bf16 64", op="layer", T=64, H=2048, E=256, I=512, shared_I=512, topk=8, scoring="softmax",
             bias=False, n_group=1, topk_group=1, scale=1.0, weights="bf16", residual=True),
        # MXFP8 weights, one token, without a shared expert
        dict(name="layer mxfp8 1", op="layer", T=1, H=2048, E=256, I=512, shared_I=0, topk=8, scoring="softmax",
             bias=False, n_group=1, topk_group=1, scale=1.0, weights="mxfp8", residual=False),
        # few wide experts in MXFP8 (K 7168, 16 experts: the benchmark's C2 widths), a wider shared expert
        dict(name="layer mxfp8 40", op="layer", T=40, H=7168, E=16, I=2048, shared_I=4096, topk=4, scoring="softmax",
             bias=False, n_group=1, topk_group=1, scale=1.0, weights="mxfp8", residual=True),
        # a projection of one token with bias and residual
        dict(name="linear 1", op="linear", M=1, N=2048, K=2048, act="none", bias=True, residual=True, out="bf16"),
        # the gated half of a wide shared expert on a decoding batch
        dict(name="linear swiglu 48", op="linear", M=48, N=2048, K=7168, act="swiglu", bias=False, residual=False,
             out="bf16"),
        # a ragged batch of prompt tokens through an ordinary feed-forward
        dict(name="linear gelu 777", op="linear", M=777, N=5125, K=1288, act="gelu_tanh", bias=True, residual=False,
             out="bf16"),
        # a long prompt chunk's down product with its residual
        dict(name="linear 8192", op="linear", M=8192, N=7168, K=4096, act="none", bias=False, residual=True,
             out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["gate", "layer", "linear"])
        if op == "linear":
            act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
            c = dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 200, 8192), K=_log_int(rng, 256, 7168), act=act,
                     bias=rng.random() < 0.5, residual=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]))
            if rng.random() < 0.85:  # rows of whole 16-byte units, as nearly every model has
                c["K"] = max(8, c["K"] // 8 * 8)
            if rng.random() < 0.5:
                c["N"] = max(64, c["N"] // 64 * 64)
            ok = c["M"] * c["N"] * c["K"] * (2 if act == "swiglu" else 1) <= 8192 * 7168 * 4096
        else:
            n_group = rng.choice([1, 1, 4, 8])
            c = dict(op=op, T=_log_int(rng, 1, 16384 if op == "gate" else 64), H=_log_int(rng, 512, 7168) // 8 * 8,
                     E=_log_int(rng, 8, 512 if op == "gate" else 256))
            c["E"] = max(c["E"] // n_group * n_group, 2 * n_group)
            scoring = rng.choice(["softmax", "sigmoid"])
            c.update(topk=rng.randint(1, min(8, c["E"] // n_group)), scoring=scoring,
                     bias=scoring == "sigmoid" and rng.random() < 0.7, n_group=n_group,
                     topk_group=rng.randint(1, n_group), scale=rng.choice([1.0, 2.5]))
            ok = c["T"] * c["H"] * max(c["E"], 64) <= 16384 * 2048 * 256
            if op == "layer":
                c.update(I=_log_int(rng, 128, 2048) // 8 * 8, weights=rng.choice(["bf16", "mxfp8"]),
                         residual=rng.random() < 0.7)
                c["shared_I"] = rng.choice([0, c["I"], 2 * c["I"]])
                used = min(c["E"], c["T"] * c["topk"])
                ok = (c["E"] + 2) * c["I"] * c["H"] <= 256 * 512 * 2048 and used * c["I"] * c["H"] <= 240 * 512 * 2048 \
                    and c["T"] * c["topk"] * c["I"] * c["H"] <= 576 * 512 * 2048
        if ok and 3072 not in c.values():
            return c


# ------------------------------------------------------------------------------------- the inputs
def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def _mx(gen, E, K, N):
    """MXFP8 weights [E, K, N] and their E8M0 scale bytes [E, ceil(K/64), N, 2] (one per 32 K)."""
    codes = torch.empty((E, K, N), dtype=torch.float8_e4m3fn, device=DEV)
    flat = codes.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):  # in pieces: the largest weights would take 4 GB in 32 bits
        flat[i:i + step] = torch.randn(min(step, flat.numel() - i), generator=gen, device=DEV).to(codes.dtype)
    e = 127 - round(math.log2(math.sqrt(K)))
    scale = torch.randint(e - 2, e + 2, (E, (K + 63) // 64, N, 2), generator=gen, device=DEV, dtype=torch.uint8)
    return codes, scale


def _scores64(case, x, wg, bias):
    """The router's scores and selection keys in 64 bits: [T, E] each, -inf keys outside the chosen groups;
    and the smallest gap, relative to the scores, between any two that have to be told apart."""
    z = x.double() @ wg.double().T
    p = torch.softmax(z, -1) if case["scoring"] == "softmax" else 1 / (1 + torch.exp(-z))
    s = p if bias is None else p + bias.double()
    gap = torch.full((x.shape[0],), float("inf"), dtype=torch.float64, device=x.device)
    g, kg = case["n_group"], case["topk_group"]
    if g > 1:
        top2 = s.view(-1, g, case["E"] // g).topk(2, -1).values.sum(-1)
        order = top2.sort(-1, descending=True).values
        if kg < g:
            gap = (order[:, kg - 1] - order[:, kg]) / order[:, kg - 1].abs()
        keep = torch.zeros_like(top2, dtype=torch.bool).scatter_(1, top2.topk(kg, -1).indices, True)
        s = s.masked_fill(~keep.repeat_interleave(case["E"] // g, 1), -float("inf"))
    order = s.topk(min(case["topk"] + 1, case["E"]), -1).values
    if order.shape[1] > 1:
        gap = torch.minimum(gap, ((order[:, :-1] - order[:, 1:]) / order[:, :-1].abs()).min(-1).values)
    return p, s, gap


def _router_inputs(case, gen):
    """Tokens after a norm, router weights and the selection bias that balances experts.  Tokens with two scores
    closer than sums in 32 bits can tell apart have no one right choice: they are left out."""
    T, H, E = case["T"], case["H"], case["E"]
    wg = _randn(gen, E, H, scale=1.3 / math.sqrt(H))
    bias = _randn(gen, E, scale=0.05, dtype=torch.float32) if case["bias"] else None
    x = _randn(gen, T + T // 8 + 16, H)
    bad = _scores64(case, x, wg, bias)[2] < 2e-5
    x = x[torch.sort(bad.to(torch.int32), dim=0, stable=True).indices[:T]].contiguous()
    return x, wg, bias


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "linear":
        rows = case["N"] * (2 if case["act"] == "swiglu" else 1)
        return dict(x=_randn(gen, case["M"], case["K"]), w=_randn(gen, rows, case["K"], scale=case["K"] ** -0.5),
                    bias=_randn(gen, rows, scale=0.3) if case["bias"] else None,
                    residual=_randn(gen, case["M"], case["N"]) if case["residual"] else None)
    x, wg, bias = _router_inputs(case, gen)
    d = dict(x=x, wg=wg, bias=bias)
    if case["op"] == "layer":
        d["residual"] = _randn(gen, case["T"], case["H"]) if case["residual"] else None
        for name, E, I in (("", case["E"], case["I"]), ("shared_", 1, case["shared_I"])):
            if I == 0:
                continue
            H = case["H"]
            if case["weights"] == "bf16":
                d[name + "w13"] = _randn(gen, E, H, 2 * I, scale=H ** -0.5)
                d[name + "w2"] = _randn(gen, E, I, H, scale=I ** -0.5)
            else:
                d[name + "w13"], d[name + "s13"] = _mx(gen, E, H, 2 * I)
                d[name + "w2"], d[name + "s2"] = _mx(gen, E, I, H)
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    st = dict(case=case, inputs=d)
    if own:
        from moe_grouped_gemm_mxfp8_gb300 import binding as B

        if case["op"] == "linear":
            # the activations' buffers and the scratch space of a program that runs this product every step
            st["call"] = B.Linear(d["w"], bias=d["bias"], activation=case["act"],
                                  out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        else:
            gate = dict(topk=case["topk"], scoring=case["scoring"], select_bias=d["bias"], n_group=case["n_group"],
                        topk_group=case["topk_group"], renormalise=True, scale=case["scale"])
            if case["op"] == "gate":
                st["call"] = B.MoeGate(d["wg"], **gate)
            else:
                # the weights laid out once, as they are when a model is loaded
                shared = case["shared_I"] > 0
                st["call"] = B.MoeLayer(
                    d["wg"], d["w13"], d["w2"], w13_scale=d.get("s13"), w2_scale=d.get("s2"),
                    shared_w13=d["shared_w13"][0] if shared else None, shared_w2=d["shared_w2"][0] if shared else None,
                    shared_w13_scale=d["shared_s13"][0] if "shared_s13" in d else None,
                    shared_w2_scale=d["shared_s2"][0] if "shared_s2" in d else None, **gate)
    return st


# ------------------------------------------------------------------------------------- the plain forms
def _plain_gate(case, d):
    z = d["x"].float() @ d["wg"].float().T
    if case["scoring"] == "softmax":
        e = torch.exp(z - z.amax(-1, keepdim=True))
        p = e / e.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-z))
    s = p if d["bias"] is None else p + d["bias"]
    g = case["n_group"]
    if g > 1:
        per = case["E"] // g
        best = torch.sort(s.view(-1, g, per), dim=-1, descending=True).values[..., :2].sum(-1)
        rank = torch.sort(best, dim=-1, descending=True, stable=True).indices
        keep = torch.zeros_like(best, dtype=torch.bool).scatter(1, rank[:, :case["topk_group"]], True)
        s = torch.where(keep.repeat_interleave(per, 1), s, torch.full_like(s, -float("inf")))
    ids = torch.sort(s, dim=-1, descending=True, stable=True).indices[:, :case["topk"]]
    w = torch.gather(p, 1, ids)
    w = w / (w.sum(-1, keepdim=True) + 1e-20) * case["scale"]
    return ids.to(torch.int32), w


def _weight32(d, name, scale, ids):
    """Weights of the chosen experts in 32 bits, [P, K, N]."""
    w = d[name][ids] if d[name].dtype == torch.bfloat16 else d[name].view(torch.uint8)[ids].view(torch.float8_e4m3fn)
    w = w.float()
    if scale in d:
        s = d[scale][ids]  # [P, ceil(K/64), N, 2]
        s = torch.exp2(s.float() - 127).permute(0, 1, 3, 2).reshape(s.shape[0], -1, s.shape[2])
        w = w * s.repeat_interleave(32, 1)[:, :w.shape[1]]
    return w


def _plain_ffn(d, prefix, ids, x):
    """x [P, n, H] through experts ids [P]: [P, n, H] in 32 bits."""
    y = x @ _weight32(d, prefix + "w13", prefix + "s13", ids)
    g, u = y.chunk(2, -1)
    return (g / (1 + torch.exp(-g)) * u) @ _weight32(d, prefix + "w2", prefix + "s2", ids)


def _plain_layer(case, d):
    ids, w = _plain_gate(case, d)
    T, k = ids.shape
    x = d["x"].float()
    y = _plain_ffn(d, "", ids.long().reshape(-1), x.repeat_interleave(k, 0)[:, None])
    out = (y.view(T, k, -1) * w[..., None]).sum(1)
    if case["shared_I"]:
        out = out + _plain_ffn(d, "shared_", torch.zeros(1, dtype=torch.long, device=DEV), x[None])[0]
    if d["residual"] is not None:
        out = out + d["residual"].float()
    return out.to(torch.bfloat16)


def _plain_linear(case, d):
    y = d["x"].float() @ d["w"].float().T
    if d["bias"] is not None:
        y = y + d["bias"].float()
    act = case["act"]
    if act == "relu":
        y = torch.where(y < 0, torch.zeros_like(y), y)
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    elif act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "swiglu":
        g, u = y.chunk(2, -1)
        y = g / (1 + torch.exp(-g)) * u
    if d["residual"] is not None:
        y = y + d["residual"].float()
    return y.to(torch.bfloat16 if case["out"] == "bf16" else torch.float32)


def run(state):
    case, d = state["case"], state["inputs"]
    if own:
        call = state["call"]
        if case["op"] == "gate":
            return call(d["x"])  # ids int32 [T, topk], weights float32 [T, topk]
        return call(d["x"], residual=d["residual"])
    if case["op"] == "gate":
        return _plain_gate(case, d)
    return _plain_layer(case, d) if case["op"] == "layer" else _plain_linear(case, d)


# ------------------------------------------------------------------------------------- the work of a pass
def work(case):
    if case["op"] == "linear":
        rows = case["N"] * (2 if case["act"] == "swiglu" else 1)
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=2 * (M * K + rows * K + (rows if case["bias"] else 0) + (M * N if case["residual"] else 0))
                    + M * N * (2 if case["out"] == "bf16" else 4), flops=2 * M * rows * K)
    T, H, E, k = case["T"], case["H"], case["E"], case["topk"]
    byte = 2 * T * H + 2 * E * H + (4 * E if case["bias"] else 0)
    flops = 2 * T * H * E
    if case["op"] == "gate":
        return dict(bytes=byte + 8 * T * k, flops=flops)
    # experts that are chosen at all: T tokens choose k of E independently
    used = E * (1 - (1 - k / E) ** T)
    wide = 2 if case["weights"] == "bf16" else 1 + 1 / 32
    byte += wide * 3 * H * (used * case["I"] + case["shared_I"]) + 2 * T * H * (2 if case["residual"] else 1)
    return dict(bytes=int(byte), flops=flops + 6 * T * H * (k * case["I"] + case["shared_I"]))


# ------------------------------------------------------------------------------------- the values in 64 bits
def _expert64(d, prefix, e):
    out = []
    for w, s in (("w13", "s13"), ("w2", "s2")):
        m = d[prefix + w][e].double()
        if prefix + s in d:
            f = torch.exp2(d[prefix + s][e].double() - 127)
            k = torch.arange(m.shape[0], device=DEV)
            m = m * f[k // 64, :, (k // 32) % 2]
        out.append(m)
    return out


def _swiglu64(y):
    n = y.shape[-1] // 2
    return y[..., :n] * torch.sigmoid(y[..., :n]) * y[..., n:]


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "linear":
        y = d["x"].double() @ d["w"].double().T
        if d["bias"] is not None:
            y += d["bias"].double()
        act = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "gelu": torch.nn.functional.gelu,
               "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
               "silu": lambda v: v * torch.sigmoid(v), "swiglu": _swiglu64}[case["act"]]
        y = act(y)
        return y if d["residual"] is None else y + d["residual"].double()
    p, s, _ = _scores64(case, d["x"], d["wg"], d["bias"])
    ids = s.topk(case["topk"], -1).indices
    w = p.gather(1, ids)
    w = w / (w.sum(-1, keepdim=True) + 1e-20) * case["scale"]
    if case["op"] == "gate":
        return None, w
    x = d["x"].double()
    out = torch.zeros_like(x) if d["residual"] is None else d["residual"].double()
    for e in ids.unique().tolist():
        t, k = (ids == e).nonzero(as_tuple=True)
        w13, w2 = _expert64(d, "", e)
        out[t] += w[t, k, None] * (_swiglu64(x[t] @ w13) @ w2)
    if case["shared_I"]:
        w13, w2 = _expert64(d, "shared_", 0)
        out += _swiglu64(x @ w13) @ w2
    return out
