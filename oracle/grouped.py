"""CPU oracles, in float64, of the products grouped by expert and the dense product with adapters.

TEST INFRASTRUCTURE ONLY.  Formulas as in include/gmmfr.h (gmmfr_grouped_linear, gmmfr_grouped_linear_grad_weight,
gmmfr_lora_linear); nothing is rounded, so each returns the exact value up to float64 arithmetic.
"""
from __future__ import annotations

import numpy as np

from oracle import moe


def grouped_linear(x, weight, sizes):
    """x [M, K], weight [E, N, K], rows of each expert.  Returns y [M, N], zeros in rows of no expert, and sum |w x|."""
    y, a = (np.zeros((x.shape[0], weight.shape[1])) for _ in range(2))
    start = 0
    for e, n in enumerate(sizes):
        at = slice(start, start + int(n))
        y[at] = x[at] @ weight[e].T
        a[at] = np.abs(x[at]) @ np.abs(weight[e]).T
        start += int(n)
    return y, a


def grouped_linear_grad_weight(dy, x, sizes):
    """dW [E, N, K] and sum |dy x|."""
    g, a = (np.zeros((len(sizes), dy.shape[1], x.shape[1])) for _ in range(2))
    start = 0
    for e, n in enumerate(sizes):
        at = slice(start, start + int(n))
        g[e] = dy[at].T @ x[at]
        a[e] = np.abs(dy[at]).T @ np.abs(x[at])
        start += int(n)
    return g, a


def lora_linear(x, w, a, b, scale, ids, bias=None, residual=None, activation="none"):
    """Returns y [M, N] and how far errors move it, per eps: of eps * sum |x w| in the product, eps * scale sum |x A| |B| in
    the adapters' sums."""
    z = x @ w.T
    absb = np.abs(x) @ np.abs(w).T
    for i in np.unique(ids):
        if 0 <= i < len(a):
            t = ids == i
            z[t] += scale[i] * ((x[t] @ a[i].T) @ b[i].T)
            absb[t] += np.abs(scale[i]) * (np.abs(x[t]) @ np.abs(a[i]).T) @ np.abs(b[i]).T
    if bias is not None:
        z = z + bias
        absb = absb + np.abs(bias)
    y = moe.ACT[activation](z)
    if activation == "swiglu":
        n = z.shape[1] // 2
        absb = 1.1 * np.abs(z[:, n:]) * absb[:, :n] + np.abs(moe.silu(z[:, :n])) * absb[:, n:]
    else:
        absb = 1.13 * absb
    return (y if residual is None else y + residual), absb
