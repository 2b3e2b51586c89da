"""silu and gelu in 64 bits, without cancellation, and what fp32 forms of them
may differ by, relative to the value.

silu(y) = y / (1 + e), e = exp(-y).  The argument of the hardware's
exponential, y log2(e), is rounded twice (the constant and the product):
|y| (2^-24 + 2^-26) of e; exponential and reciprocal are within 2^-23 of
theirs, the sum and the product within 2^-24: |y| 2^-23 + 2^-21 of silu(y).
Where 1 + e passes 2^126 its reciprocal is below the normal numbers and may be
0: y 2^-126.

gelu(y) = y erfc(-y / sqrt 2) / 2.  erfc is a polynomial of 1 / (1 + p |y|)
times exp(-y^2 / 2).  The argument of the exponential is rounded twice and its
constant once, y^2 / 2 (2^-23 + 2^-26) of e, and the polynomial is within
2^-25 (1 + y^2 / 2) of its function: together y^2 2^-23.  The roundings of the
polynomial's argument (2^-24, 2^-23) move it by less than themselves, its
eight steps add their 2^-24 (2.2 times its size of terms, each step half that
of the last): 7 2^-24; the exponential and three products 5 2^-24.  With 1 -
erfc / 2 for y > 0 the same is smaller: 2^-20 + y^2 2^-23 of gelu(y).  An
exponential below the normal numbers may be 0: the rest of y erfc / 2 is below
1 there, 2^-126."""
from math import erfc

import numpy as np

SLOPE = 1.13       # of both, at most


def silu(y):
    with np.errstate(over="ignore"):
        return y / (1 + np.exp(-y))


def gelu(y):
    return y * 0.5 * np.vectorize(erfc, otypes=[float])(-y / np.sqrt(2.0))


def activate(y, dy, act):
    """(value, bound) for finite sums y known within dy."""
    if act == "none":
        return y, dy
    if act == "silu":
        v = silu(y)
        return v, SLOPE * dy + (2.0 ** -21 + np.abs(y) * 2.0 ** -23) * np.abs(v) + np.abs(y) * 2.0 ** -126
    if act == "gelu":
        v = gelu(y)
        return v, SLOPE * dy + (2.0 ** -20 + y * y * 2.0 ** -23) * np.abs(v) + 2.0 ** -126
    n = y.shape[1] // 2
    s, ds = activate(y[:, :n], dy[:, :n], "silu")
    u, du = y[:, n:], dy[:, n:]
    return s * u, ds * (np.abs(u) + du) + np.abs(s) * du + 2.0 ** -23 * np.abs(s * u)


def product(w, x, act="none", bias=None, residual=None):
    """w [n, k], x [rows, k] float64 -> (value, bound before the output's
    rounding).  The sums: product_ref."""
    y, a = x @ w.T, np.abs(x) @ np.abs(w).T
    b = np.zeros(w.shape[0]) if bias is None else bias
    y = y + b
    dy = (w.shape[1] + 1) * 2.0 ** -23 * a + 2.0 ** -23 * (np.abs(y) + np.abs(b))
    v, dv = activate(y, dy, act)
    if residual is not None:
        v = v + residual
        dv = dv + 2.0 ** -24 * (np.abs(v) + np.abs(residual) + dv)
    return v, dv
