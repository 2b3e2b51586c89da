"""Plain 64-bit forms of the route lists, the grouped and the dense products,
with bounds on what fp32 sums may differ by.  numpy only, from the
definitions; shares nothing with the library.

Bounds.  The products of two bf16 values are exact in fp32; a sum of k of
them in any order is within k 2^-23 of the sum of their magnitudes A (one
rounding, or one truncation, each).  An E2M1 matrix's global scale adds one
rounding, the bias another: dy = k 2^-23 A + 2^-23 (|y| + |bias|).  silu and
gelu have slopes below 1.13, and are evaluated within 2^-20 |y| (exp, erf and
a division of a few roundings each; 1 + erf loses its leading bits, which
costs an absolute 2^-22 times |y| / 2).  The output is rounded once."""
import numpy as np

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133}   # steps below the normal numbers


def lists(idx, P):
    flat = np.asarray(idx).reshape(-1)
    buckets = [[] for _ in range(P + 1)]
    for r, e in enumerate(flat.tolist()):
        buckets[e if 0 <= e < P else P].append(r)
    offsets = np.cumsum([0] + [len(b) for b in buckets[:P]])
    return offsets.astype(np.int32), np.array([r for b in buckets for r in b], np.int32)


def _silu(y):
    with np.errstate(over="ignore"):
        return y / (1 + np.exp(-y))


def _gelu(y):
    from math import erf

    return y * 0.5 * (1 + np.vectorize(erf, otypes=[float])(y / np.sqrt(2.0)))


def activate(y, dy, act):
    """(value, bound) of the activation of sums y known within dy."""
    if act == "none":
        return y, dy
    if act in ("silu", "gelu"):
        return (_silu(y) if act == "silu" else _gelu(y)), 1.13 * dy + 2.0 ** -20 * np.abs(y)
    n = y.shape[1] // 2
    g, u, dg, du = y[:, :n], y[:, n:], dy[:, :n], dy[:, n:]
    s = _silu(g)
    ds = 1.13 * dg + 2.0 ** -20 * np.abs(s)
    return s * u, ds * (np.abs(u) + du) + np.abs(s) * du + 2.0 ** -23 * np.abs(s * u)


def product(w, x, act="none", bias=None, residual=None):
    """w [n, k], x [rows, k] float64 -> (value, bound before the output's rounding)."""
    y, a = x @ w.T, np.abs(x) @ np.abs(w).T
    b = np.zeros(w.shape[0]) if bias is None else bias
    y = y + b
    dy = (w.shape[1] + 1) * 2.0 ** -23 * a + 2.0 ** -23 * (np.abs(y) + np.abs(b))
    v, dv = activate(y, dy, act)
    if residual is not None:
        v = v + residual
        dv = dv + 2.0 ** -24 * (np.abs(v) + np.abs(residual) + dv)
    return v, dv


def grouped(w, x, offsets, out_rows, matrices=None, gather=None, div=1, scatter=None, R=None, act="none", bias=None):
    """w [P, n, k]; returns (written [out_rows], value, bound)."""
    P, n = w.shape[:2]
    cols = n // 2 if act == "swiglu" else n
    R = len(x) if R is None else R
    done = np.zeros(out_rows, bool)
    val, bnd = np.zeros((out_rows, cols)), np.zeros((out_rows, cols))
    for g in range(len(offsets) - 1):
        m = g if matrices is None else int(matrices[g])
        places = [i for i in range(max(int(offsets[g]), 0), min(int(offsets[g + 1]), R))]
        src = [int(i if gather is None else (gather[i] // div if gather[i] >= 0 else -1)) for i in places]
        dst = [int(i if scatter is None else scatter[i]) for i in places]
        pairs = [(s, d) for s, d in zip(src, dst) if 0 <= s < len(x) and 0 <= d < out_rows]
        if not pairs:
            continue
        s, d = np.array(pairs).T
        done[d] = True
        if 0 <= m < P:
            val[d], bnd[d] = product(w[m], x[s], act, None if bias is None else bias[m])
    return done, val, bnd


def off(got, val, bnd, dtype):
    """The largest excess over the bound and half a step of the output's type (<= 0: fine)."""
    half = HALF[dtype]
    return float((np.abs(got - val) - (bnd * (1 + half) + np.abs(val) * half + TINY[dtype])).max(initial=-np.inf))
