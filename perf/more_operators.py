"""Measured cases of the products whose rows belong to different weights: products grouped by expert, with their
gradients (``grouped``), and the dense product with low-rank adapters of many requests (``lora``).

Each case runs in two forms on the same inputs: ``own = False`` computes the operator with
elementary torch operations in 32 bits, rounded once at the end; ``own = True`` makes the calls a
user makes of the library.  ``exact`` gives the definition's value in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"

DIRECTIONS = ("y", "dx", "dw", "step")


# ------------------------------------------------------------------------------------- the cases
def _grouped(name, M, E, K, N, direction, groups="random", transposed=False, out="bf16", rest=0):
    return dict(name=name, op="grouped", M=M, E=E, K=K, N=N, direction=direction, groups=groups, transposed=transposed,
                out=out, rest=rest)


def _lora(name, M, N, K, L, r, act="none", bias=False, residual=False, rows="tokens", out="bf16"):
    return dict(name=name, op="lora", M=M, N=N, K=K, L=L, r=r, act=act, bias=bias, residual=residual, rows=rows, out=out)


def listed():
    return [
        # one decoded token's eight experts through their gate and up weights (LLaDA2.0-mini: 256 experts, H 2048, I 512)
        _grouped("grouped y 8", 8, 256, 2048, 1024, "y", groups="distinct", transposed=True),
        # a decoding batch of 64 tokens, top-8: most experts have a few rows, some none
        _grouped("grouped y 512", 512, 256, 2048, 1024, "y", transposed=True),
        # prompts' tails through few wide experts (K 7168: the benchmark's C2 widths), popular experts first, FP32 results
        _grouped("grouped y 3001", 3001, 16, 7168, 1544, "y", groups="zipf", out="f32"),
        # gradient of the rows of a small training batch: 16 rows an expert
        _grouped("grouped dx 4096", 4096, 256, 512, 2048, "dx"),
        # gradient of the weights of the same batch: the writing of them
        _grouped("grouped dw 4096", 4096, 256, 2048, 1024, "dw", transposed=True),
        # gradient of the weights in FP32, few experts of uneven popularity, rows behind the last group
        _grouped("grouped dw 9999", 9999, 24, 5120, 1288, "dw", groups="zipf", out="f32", rest=77),
        # a training step's forward and both gradients, 8192 tokens top-8 over 64 experts
        _grouped("grouped step 65536", 65536, 64, 2048, 1024, "step"),
        # one request's decoded token with its adapter
        _lora("lora 1", 1, 2048, 2048, 64, 16),
        # a decoding batch, nearly every request with an adapter of its own
        _lora("lora 48", 48, 4096, 4096, 64, 16, residual=True),
        # the gated half of a feed-forward, larger ranks, few adapters
        _lora("lora swiglu 100", 100, 2048, 7168, 8, 64, act="swiglu", bias=True),
        # ends of prompts and decoded tokens in one batch
        _lora("lora gelu 777", 777, 5125, 1288, 32, 32, act="gelu_tanh", bias=True, rows="mixed"),
        # a long prompt chunk of a few requests, each with its adapter
        _lora("lora 8192", 8192, 7168, 4096, 16, 16, residual=True, rows="prompts"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        if rng.random() < 0.55:
            c = dict(op="grouped", M=_log_int(rng, 1, 65536), E=_log_int(rng, 1, 512), K=_log_int(rng, 128, 7168) // 8 * 8,
                     N=_log_int(rng, 128, 7168) // 8 * 8, direction=rng.choice(DIRECTIONS),
                     groups=rng.choice(["random", "random", "zipf"]), transposed=rng.random() < 0.5,
                     out=rng.choice(["bf16", "bf16", "f32"]), rest=rng.choice([0, 0, 0, rng.randint(1, 300)]))
            ok = c["E"] * c["N"] * c["K"] <= 256 * 2048 * 1024 and c["M"] * c["N"] * c["K"] <= 65536 * 2048 * 1024 \
                and c["M"] * (c["N"] + c["K"]) <= 65536 * 5120
        else:
            c = dict(op="lora", M=_log_int(rng, 1, 8192), N=_log_int(rng, 200, 8192), K=_log_int(rng, 256, 7168) // 8 * 8,
                     L=_log_int(rng, 1, 256), r=rng.choice([8, 16, 16, 24, 32, 64, 128]),
                     act=rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"]),
                     bias=rng.random() < 0.5, residual=rng.random() < 0.5, rows=rng.choice(["tokens", "mixed", "prompts"]),
                     out=rng.choice(["bf16", "bf16", "f32"]))
            if rng.random() < 0.5:
                c["N"] = max(64, c["N"] // 64 * 64)
            wide = 2 if c["act"] == "swiglu" else 1
            ok = c["M"] * c["N"] * c["K"] * wide <= 8192 * 7168 * 4096 and c["L"] * c["r"] <= 8192 \
                and c["N"] * c["K"] * wide <= 8192 * 5120
        if ok:
            return c


# ------------------------------------------------------------------------------------- the inputs
def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat, step = out.view(-1), 1 << 28  # in pieces: the largest weights would take 2 GB in 32 bits
    for i in range(0, flat.numel(), step):
        flat[i:i + step] = torch.randn(min(step, flat.numel() - i), generator=gen, device=DEV) * scale
    return out


def _group_sizes(case, host):
    """Rows of each expert: M - rest in all, in the order of the experts."""
    M, E = case["M"] - min(case["rest"], case["M"] - 1), case["E"]
    if case["groups"] == "distinct":  # as many experts as rows, one row each
        chosen = torch.randperm(E, generator=host)[:M]
        return torch.zeros(E, dtype=torch.int64).index_add_(0, chosen, torch.ones_like(chosen))
    weight = torch.ones(E, dtype=torch.float64)
    if case["groups"] == "zipf":
        weight = 1 / torch.arange(1, E + 1, dtype=torch.float64)
        weight = weight[torch.randperm(E, generator=host)]
    chosen = torch.multinomial(weight, M, replacement=True, generator=host)
    return torch.bincount(chosen, minlength=E)


def _adapter_rows(case, host):
    """The adapter of each row, -1 for none."""
    M, L = case["M"], case["L"]
    ids = torch.randint(0, L, (M,), generator=host)
    ids[torch.rand(M, generator=host) < 0.1] = -1
    if case["rows"] == "tokens":  # every row another request's
        if M == 1:
            ids = torch.randint(0, L, (1,), generator=host)
        return ids.to(torch.int32)
    # requests' prompts one after the other; "mixed": behind them an eighth of the rows are decoded tokens
    at, end = 0, M if case["rows"] == "prompts" else M - M // 8
    while at < end:
        n = int(torch.randint(1, max(2, M // 4), (1,), generator=host))
        ids[at:min(at + n, end)] = ids[at].item()
        at += n
    return ids.to(torch.int32)


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    if case["op"] == "grouped":
        M, E, K, N = case["M"], case["E"], case["K"], case["N"]
        sizes = _group_sizes(case, host)
        d = dict(group_list=sizes.to(DEV), ends=[0] + sizes.cumsum(0).tolist())
        d["weight"] = _randn(gen, *((E, K, N) if case["transposed"] else (E, N, K)), scale=K ** -0.5)
        if case["direction"] != "dx":
            d["x"] = _randn(gen, M, K)
        if case["direction"] != "y":
            d["dy"] = _randn(gen, M, N, scale=0.02)  # gradients of a mean over the rows are small
        return d
    M, N, K, L, r = case["M"], case["N"], case["K"], case["L"], case["r"]
    rows = N * (2 if case["act"] == "swiglu" else 1)
    d = dict(x=_randn(gen, M, K), weight=_randn(gen, rows, K, scale=K ** -0.5), a=_randn(gen, L, r, K, scale=K ** -0.5),
             b=_randn(gen, L, rows, r, scale=0.5 * r ** -0.5), ids=_adapter_rows(case, host).to(DEV))
    # alpha / rank, alpha between r / 2 and 2 r
    d["scale"] = torch.exp2(torch.rand(L, generator=gen, device=DEV) * 2 - 1)
    d["bias"] = _randn(gen, rows, scale=0.3) if case["bias"] else None
    d["residual"] = _randn(gen, M, N) if case["residual"] else None
    return d


def _dtype(case):
    return torch.bfloat16 if case["out"] == "bf16" else torch.float32


def prepare(case, seed):
    d = _inputs(case, seed)
    st = dict(case=case, inputs=d)
    if own:
        from moe_grouped_gemm_mxfp8_gb300 import binding as B

        if case["op"] == "grouped":
            st["call"] = B.GroupedLinear(d["weight"], transposed=case["transposed"], out_dtype=_dtype(case),
                                         grad_dtype=_dtype(case))
        else:
            st["call"] = B.LoraLinear(d["weight"], d["a"], d["b"], scale=d["scale"], bias=d["bias"], activation=case["act"],
                                      out_dtype=_dtype(case))
    return st


# ------------------------------------------------------------------------------------- the plain forms
def _plain_grouped(case, d):
    """Expert after expert, the groups' ends known to the program.  Rows behind the last group are zeros."""
    out, step, ends = _dtype(case), case["direction"] == "step", d["ends"]
    weight = d["weight"]
    res = {}
    if step or case["direction"] == "y":
        res["y"] = torch.zeros((case["M"], case["N"]), dtype=out, device=DEV)
    if step or case["direction"] == "dx":
        res["dx"] = torch.zeros((case["M"], case["K"]), dtype=torch.bfloat16, device=DEV)
    if step or case["direction"] == "dw":
        res["dw"] = torch.zeros(weight.shape, dtype=out, device=DEV)
    for e in range(case["E"]):
        at = slice(ends[e], ends[e + 1])
        if at.start == at.stop:
            continue
        if "y" in res or "dx" in res:
            w = weight[e].float()  # [N, K], or [K, N]
        if "y" in res:
            res["y"][at] = (d["x"][at].float() @ (w if case["transposed"] else w.T)).to(out)
        if "dx" in res:
            res["dx"][at] = (d["dy"][at].float() @ (w.T if case["transposed"] else w)).to(torch.bfloat16)
        if "dw" in res:
            left, right = (d["x"], d["dy"]) if case["transposed"] else (d["dy"], d["x"])
            res["dw"][e] = (left[at].float().T @ right[at].float()).to(out)
    return res


def _activated(act, y):
    if act == "relu":
        return torch.where(y < 0, torch.zeros_like(y), y)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "swiglu":
        g, u = y.chunk(2, -1)
        return g / (1 + torch.exp(-g)) * u
    return y


def _plain_lora(case, d):
    """Every row through all adapters' first factors and its own second one: the rows' own sums are selected by
    comparison, so that nothing waits for the host to learn which adapters there are."""
    x = d["x"].float()
    y = x @ d["weight"].float().T
    if d["bias"] is not None:
        y = y + d["bias"].float()
    L, r, K = d["a"].shape
    s = (x @ d["a"].float().view(L * r, K).T).view(-1, L, r)
    s = s * d["scale"][None, :, None]
    mine = d["ids"][:, None] == torch.arange(L, dtype=torch.int32, device=DEV)[None]
    s = torch.where(mine[..., None], s, torch.zeros_like(s))
    b = d["b"].float()  # [L, rows, r]
    y = y + s.view(-1, L * r) @ b.permute(0, 2, 1).reshape(L * r, -1)
    y = _activated(case["act"], y)
    if d["residual"] is not None:
        y = y + d["residual"].float()
    return y.to(_dtype(case))


def run(state):
    case, d = state["case"], state["inputs"]
    if not own:
        return _plain_grouped(case, d) if case["op"] == "grouped" else _plain_lora(case, d)
    call = state["call"]
    if case["op"] == "lora":
        return call(d["x"], d["ids"], residual=d["residual"])
    step, groups, res = case["direction"] == "step", d["group_list"], {}
    if step or case["direction"] == "y":
        res["y"] = call(d["x"], groups)
    if step or case["direction"] == "dx":
        res["dx"] = call.grad_input(d["dy"], groups)
    if step or case["direction"] == "dw":
        res["dw"] = call.grad_weight(d["dy"], d["x"], groups)
    return res


# ------------------------------------------------------------------------------------- the work of a pass
def work(case):
    wide = 2 if case["out"] == "bf16" else 4
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "grouped":
        E, rows = case["E"], M - min(case["rest"], M - 1)
        # experts that have rows at all
        if case["groups"] == "distinct":
            used = min(E, rows)
        elif case["groups"] == "random":
            used = E * (1 - (1 - 1 / E) ** rows)
        else:
            total = sum(1 / i for i in range(1, E + 1))
            used = sum(1 - (1 - 1 / (i * total)) ** rows for i in range(1, E + 1))
        n = 3 if case["direction"] == "step" else 1
        byte = 8 * E
        if case["direction"] in ("y", "step"):
            byte += M * N * wide
        if case["direction"] in ("dx", "step"):
            byte += 2 * M * K
        if case["direction"] in ("dw", "step"):
            byte += wide * E * N * K
        if case["direction"] != "dw":
            byte += 2 * used * N * K
        if case["direction"] != "dx":
            byte += 2 * rows * K
        if case["direction"] != "y":
            byte += 2 * rows * N
        return dict(bytes=int(byte), flops=2 * n * rows * N * K)
    L, r = case["L"], case["r"]
    rows_w = N * (2 if case["act"] == "swiglu" else 1)
    # adapters that any row has: requests have their rows together, about eight rows or pieces of a batch
    requests = M if case["rows"] == "tokens" else (8 if case["rows"] == "prompts" else 8 + M // 8)
    used = L * (1 - (1 - 1 / L) ** min(M, requests))
    byte = 2 * (M * K + rows_w * K + (rows_w if case["bias"] else 0) + (M * N if case["residual"] else 0)) + M * N * wide
    byte += used * 2 * r * (K + rows_w) + 4 * M + 4 * L
    return dict(bytes=int(byte), flops=2 * M * rows_w * K + 2 * M * r * (K + rows_w))


# ------------------------------------------------------------------------------------- the values in 64 bits
def _exact_grouped(case, d):
    x, dy = d.get("x"), d.get("dy")
    want = ("y", "dx", "dw") if case["direction"] == "step" else (case["direction"],)
    M, K, N = case["M"], case["K"], case["N"]
    shapes = dict(y=(M, N), dx=(M, K), dw=tuple(d["weight"].shape))
    res = {k: torch.zeros(shapes[k], dtype=torch.float64, device=DEV) for k in want}
    expert = torch.bucketize(torch.arange(M), torch.tensor(d["ends"][1:]), right=True)
    for e in range(case["E"]):
        t = (expert == e).nonzero()[:, 0].to(DEV)
        if not len(t):
            continue
        w = d["weight"][e].double()
        w = w.mT if case["transposed"] else w  # [N, K]
        if "y" in res:
            res["y"].index_copy_(0, t, torch.einsum("tk,nk->tn", x[t].double(), w))
        if "dx" in res:
            res["dx"].index_copy_(0, t, torch.einsum("tn,nk->tk", dy[t].double(), w))
        if "dw" in res:
            g = torch.einsum("tn,tk->nk", dy[t].double(), x[t].double())
            res["dw"][e] = g.mT if case["transposed"] else g
    return res


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "grouped":
        return _exact_grouped(case, d)
    x = d["x"].double()
    y = x @ d["weight"].double().mT
    if d["bias"] is not None:
        y += d["bias"].double()
    for a in d["ids"].unique().tolist():
        if a >= 0:
            t = (d["ids"] == a).nonzero()[:, 0]
            y[t] += d["scale"][a].double() * ((x[t] @ d["a"][a].double().mT) @ d["b"][a].double().mT)
    act = case["act"]
    if act == "swiglu":
        n = y.shape[1] // 2
        y = y[:, :n] * torch.sigmoid(y[:, :n]) * y[:, n:]
    elif act != "none":
        y = {"relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
             "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act](y)
    return y if d["residual"] is None else y + d["residual"].double()
