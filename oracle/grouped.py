"""CPU oracles, in float64, of the products grouped by expert and the dense product with adapters.

TEST INFRASTRUCTURE ONLY.  Formulas as in include/gmmfr.h (gmmfr_grouped_linear, gmmfr_grouped_linear_grad_weight); nothing is
rounded, so each returns the exact value up to float64 arithmetic.
"""
from __future__ import annotations

import numpy as np


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
