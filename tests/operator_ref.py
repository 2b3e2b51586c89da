"""Plain 64-bit forms of the scored router, the 4-bit rows and the MXFP4
product, for the tests: written from the definitions, numpy only, sharing
nothing with the library.

Comparisons of exact values: a middle of two codes times a block scale times
a global scale has at most 31 significant bits and is exact in float64."""
import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def route(logits, K, *, score, groups=1, top_groups=1, top2=False, renorm=True, scale=1.0, bias=None):
    """logits float64 [T, E] -> (ids int32 [T, K], w float64 [T, K])."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids = np.full((T, K), -1, np.int32)
    w = np.zeros((T, K))
    gs = E // groups
    for t in range(T):
        l = logits[t]
        live = [e for e in range(E) if not np.isnan(l[e]) and l[e] != -np.inf]
        s = np.zeros(E)
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                s[live] = 1.0 / (1.0 + np.exp(-l[live]))
            elif live:
                top = max(l[live])
                ex = np.array([1.0 if l[e] == top else np.exp(l[e] - top) for e in live])
                s[live] = ex / ex.sum()
        c = l.copy() if bias is None else s + bias
        live = [e for e in live if not np.isnan(c[e]) and c[e] != -np.inf]
        per = s if (bias is None and top2) else c
        value = {}
        for g in range(groups):
            best = sorted((per[e] for e in live if e // gs == g), reverse=True)
            if best:
                value[g] = sum(best[:2]) if top2 else best[0]
        kept = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
        if groups > 1:
            live = [e for e in live if e // gs in kept]
        picks = sorted(live, key=lambda e: (-c[e], e))[:K]
        if not picks:
            continue
        sw = s[picks]
        if renorm:
            sw = sw / sw.sum() if sw.sum() > 0 else np.full(len(picks), 1.0 / len(picks))
        ids[t, :len(picks)] = picks
        w[t, :len(picks)] = sw * np.float64(np.float32(scale))
    return ids, w


def _nearest_even(ax, grid, unit):
    """Index into grid of the value nearest to ax / unit (ties to the even index), exactly."""
    idx = np.zeros(ax.shape, np.int64)
    for i in range(len(grid) - 1):
        mid = (grid[i] + grid[i + 1]) / 2 * unit
        idx += (ax > mid) if i % 2 == 0 else (ax >= mid)
    return idx


def e4m3_grid():
    b = np.arange(127)
    e, m = b // 8, b % 8
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.astype(float) - 7))


def quantize(x, fmt, glob=None, per=1):
    """x float64 [R, C] -> (codes uint8 [R, C/2], scales uint8, values float64 [R, C], NaN where the
    block's scale is)."""
    R, C = x.shape
    B = 32 if fmt == "mxfp4" else 16
    b = x.reshape(R, C // B, B)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        finite = np.isfinite(b).all(2)
        safe = np.where(finite[:, :, None], b, 0.0)
        amax = np.abs(safe).max(2)
        if fmt == "mxfp4":
            e = np.where(amax > 0, np.frexp(amax)[1] - 3, -127)
            sc = np.maximum(e + 127, 0)
            unit = np.ldexp(1.0, sc - 127)
            bad, nan = ~finite, 0xFF
            size = unit
        else:
            g = np.ones(R) if glob is None else np.asarray(glob, np.float64)[np.arange(R) // per]
            ok = (g > 0) & np.isfinite(g)
            bad, nan = ~finite | ~ok[:, None], 0x7F
            gg = np.where(ok, g, 1.0)[:, None]
            sc = _nearest_even(amax, e4m3_grid(), 6 * gg)
            unit = e4m3_grid()[sc] * gg
            size = unit
    code = _nearest_even(np.abs(safe), VALUES, size[:, :, None])
    code = np.where((unit > 0)[:, :, None] & ~bad[:, :, None], code | (np.signbit(safe).astype(int) << 3), 0)
    vals = VALUES[code & 7] * np.where(code & 8, -1.0, 1.0) * unit[:, :, None]
    vals = np.where(bad[:, :, None], np.nan, vals)
    sc = np.where(bad, nan, sc).astype(np.uint8)
    code = code.reshape(R, C).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), sc, vals.reshape(R, C)


def decode_mxfp4(codes, scales):
    """codes uint8 [.., C/2], scales uint8 [.., C/32] -> float64 [.., C]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = VALUES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def product(codes, scales, xq, idx, swiglu=False):
    """W codes [P, n, k/2], scales; xq float64 [T, k]; idx [T, K].  Returns (out, sums of magnitudes of
    the products) float64 [T*K, n or n/2]; with swiglu the second is (sum_gate, sum_up, gate, up)."""
    P, n = codes.shape[:2]
    T, K = idx.shape
    y = np.zeros((T * K, n))
    a = np.zeros((T * K, n))
    rows = idx.reshape(-1)
    for i in np.unique(rows):
        if 0 <= i < P:
            r = np.nonzero(rows == i)[0]
            w = decode_mxfp4(codes[i], scales[i])
            y[r] = xq[r // K] @ w.T
            a[r] = np.abs(xq[r // K]) @ np.abs(w).T
    if not swiglu:
        return y, a
    g, u = y[:, :n // 2], y[:, n // 2:]
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u, (a[:, :n // 2], a[:, n // 2:], g, u)
