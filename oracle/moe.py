"""CPU oracles, in float64, of the router, the few-token MoE layer and the dense product.

TEST INFRASTRUCTURE ONLY.  Formulas as in include/gmmfr.h (gmmfr_moe_gate, gmmfr_moe_layer,
gmmfr_linear); nothing is rounded, so each returns the exact value up to float64 arithmetic.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.ffn import silu

_NONE = -np.inf


def gate_probabilities(logits, scoring: str):
    z = np.asarray(logits, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        mx = z.max(-1, keepdims=True)
        e = np.where(mx == -np.inf, 0.0, np.exp(z - mx))
        s = e.sum(-1, keepdims=True)
        return np.where(s == 0.0, 0.0, e / np.where(s == 0.0, 1.0, s))


def _descending(s):
    """Indices by descending value, NaN last, equal values by index."""
    return sorted(range(len(s)), key=lambda i: (math.isnan(s[i]), 0.0 if math.isnan(s[i]) else -s[i], i))


def gate_select(logits, topk, scoring="softmax", select_bias=None, n_group=1, topk_group=1, group_top=2,
                renormalise=True, scale=1.0):
    """ids [T, topk], weights [T, topk], and the selection scores [T, E] (-inf outside eligible groups)."""
    p = gate_probabilities(logits, scoring)
    s = p if select_bias is None else p + np.asarray(select_bias, dtype=np.float64)
    s = s.copy()
    T, E = s.shape
    per = E // n_group
    ids = np.zeros((T, topk), dtype=np.int64)
    for t in range(T):
        if n_group > 1:
            score = []
            for g in range(n_group):
                v = s[t, g * per:(g + 1) * per]
                v = np.sort(np.where(np.isnan(v), -np.inf, v))[::-1]
                with np.errstate(invalid="ignore"):
                    score.append(float(v[:group_top].sum()))
            keep = _descending(score)[:topk_group]
            for g in range(n_group):
                if g not in keep:
                    s[t, g * per:(g + 1) * per] = _NONE
            eligible = [e for e in range(E) if e // per in keep]
        else:
            eligible = list(range(E))
        order = _descending([s[t, e] for e in eligible])
        ids[t] = [eligible[i] for i in order[:topk]]
    w = np.take_along_axis(p, ids, 1)
    if renormalise:
        w = w / (w.sum(-1, keepdims=True) + 1e-20)
    return ids, w * scale, s


def mx_values(codes, scale):
    """E4M3 codes [E, K, N] (uint8) with E8M0 scales [E, ceil(K/64), N, 2] -> float64 values."""
    c = np.asarray(codes).astype(np.int64)
    sign, e, m = np.where(c & 128, -1.0, 1.0), (c >> 3) & 15, (c & 7).astype(np.float64)
    v = sign * np.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * 2.0 ** (e - 7.0))
    k = np.arange(c.shape[1])
    return v * 2.0 ** (np.asarray(scale).astype(np.float64)[:, k // 64, :, (k // 32) % 2].transpose(1, 0, 2) - 127.0)


def _swiglu(y):
    n = y.shape[-1] // 2
    return silu(y[..., :n]) * y[..., n:]


def moe_layer(x, ids, weights, w13, w2, shared_w13=None, shared_w2=None, residual=None):
    """All float64.  Returns out [T, H] and absb: the sum of |weight * sw * w2| over its terms."""
    T, H = x.shape
    out = np.zeros((T, H)) if residual is None else residual.copy()
    absb = np.zeros((T, H))
    for t in range(T):
        for e, w in zip(ids[t], weights[t]):
            sw = _swiglu(x[t] @ w13[e]) * w
            out[t] += sw @ w2[e]
            absb[t] += np.abs(sw) @ np.abs(w2[e])
    if shared_w13 is not None:
        sw = _swiglu(x @ shared_w13)
        out += sw @ shared_w2
        absb += np.abs(sw) @ np.abs(shared_w2)
    return out, absb


_erf = np.vectorize(math.erf, otypes=[np.float64])
ACT = {
    "none": lambda v: v,
    "relu": lambda v: np.where(v < 0, 0.0, v),
    "gelu": lambda v: 0.5 * v * (1 + _erf(v / math.sqrt(2))),
    "gelu_tanh": lambda v: 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))),
    "silu": silu,
    "swiglu": _swiglu,
}


def linear(x, w, bias=None, residual=None, activation="none"):
    """All float64.  Returns y [M, N] and how far an error of eps * sum |x w| in every sum can move it, per eps."""
    z = x @ w.T
    a = np.abs(x) @ np.abs(w).T
    if bias is not None:
        z = z + bias
        a = a + np.abs(bias)
    y = ACT[activation](z)
    if activation == "swiglu":
        n = z.shape[1] // 2
        g, u = z[:, :n], z[:, n:]
        a = 1.1 * np.abs(u) * a[:, :n] + np.abs(silu(g)) * a[:, n:]  # |silu'| < 1.1
    else:
        a = 1.13 * a  # |gelu'| < 1.13, the largest slope of the activations
    return (y if residual is None else y + residual), a
