"""Timing cases of the scored router, the 4-bit row formats and the MXFP4
product over pool rows.

With `own` false, run() computes each operator in plain torch operations
(32-bit floats, 64 where an order or a rounding border hangs on it); with
`own` true it makes the library calls a decode program makes.  exact() is the
definition in 64 bits.

  route    scored top-K routing: softmax or sigmoid scores, a balance bias,
           expert groups, renormalised and scaled weights, masked experts
  rows     rows of floats to a 4-bit bank format and back
  product  one activation row per token, quantised to MXFP4, times the MXFP4
           matrices its routes name
"""
import math

import numpy as np
import torch

own = False

MXFP4, E2M1 = "mxfp4", "e2m1"
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token of a grouped sigmoid router with a balance bias (256 experts, top 8)
        dict(name="route-token", op="route", T=1, E=256, K=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top2=True, renorm=True, scale=2.5, dtype="float32", masked=False),
        # a ragged batch over 160 experts, bf16 logits, group maxima, raw softmax weights, some
        # experts masked out and some rows without any expert (padding rows)
        dict(name="route-batch", op="route", T=77, E=160, K=6, score="softmax", bias=False, groups=8,
             top_groups=3, group_top2=False, renorm=False, scale=16.0, dtype="bfloat16", masked=True),
        # a long prompt over 512 experts, top 10, balance bias
        dict(name="route-prompt", op="route", T=16384, E=512, K=10, score="sigmoid", bias=True, groups=1,
             top_groups=1, group_top2=False, renorm=True, scale=1.0, dtype="float32", masked=False),
        # one activation row of the 2048-wide decode
        dict(name="rows-token", op="rows", fmt=MXFP4, rows=1, cols=2048, stride=2048, per_global=0,
             dtype="bfloat16"),
        # odd rows cut out of a wider fp32 buffer, a global scale per 111 rows
        dict(name="rows-odd", op="rows", fmt=E2M1, rows=333, cols=1056, stride=1061, per_global=111,
             dtype="float32"),
        # loading 64 experts' gate/up matrices of the 2048-wide decode
        dict(name="rows-experts-mxfp4", op="rows", fmt=MXFP4, rows=65536, cols=2048, stride=2048,
             per_global=0, dtype="bfloat16"),
        # loading 16 experts' gate/up matrices of the 4096-wide prompt chunks, a global scale each
        dict(name="rows-experts-e2m1", op="rows", fmt=E2M1, rows=32768, cols=4096, stride=4096,
             per_global=2048, dtype="bfloat16"),
        # one token's gate/up over its 8 experts' rows (256 experts, H 2048, F 512)
        dict(name="product-token", op="product", T=1, K=8, pool=256, n=1024, k=2048, swiglu=True,
             out="bfloat16", skip=0.0),
        # the wide decode step: 600 rows, top 2 of 160 experts, H 1024, F 256
        dict(name="product-wide", op="product", T=600, K=2, pool=160, n=512, k=1024, swiglu=True,
             out="bfloat16", skip=0.0),
        # odd sizes, fp32 output, a tenth of the routes without a row
        dict(name="product-odd", op="product", T=45, K=3, pool=24, n=515, k=1056, swiglu=False,
             out="float32", skip=0.1),
        # a prompt through the 256 experts of the 4096-wide layer, top 6 (F 1024)
        dict(name="product-prompt", op="product", T=4096, K=6, pool=256, n=2048, k=4096, swiglu=True,
             out="bfloat16", skip=0.0),
        # one dense matrix for every row of a long prompt
        dict(name="product-dense", op="product", T=8192, K=1, pool=1, n=4096, k=4096, swiglu=False,
             out="bfloat16", skip=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("route", "rows", "product"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8, 16))
        E = groups * _log(rng, 3, 512 // groups)
        top_groups = rng.randint(1, groups)
        K = rng.randint(1, min(16, E))
        return dict(op=op, T=_log(rng, 1, 16384), E=E, K=K, score=rng.choice(("softmax", "sigmoid")),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                    group_top2=rng.random() < 0.5, renorm=rng.random() < 0.6,
                    scale=rng.choice((1.0, 2.5, 16.0)), dtype=rng.choice(("float32", "bfloat16")),
                    masked=rng.random() < 0.4)
    if op == "rows":
        fmt = rng.choice((MXFP4, E2M1))
        blk = 32 if fmt == MXFP4 else 16
        cols = blk * _log(rng, 1, 8192 // blk)
        rows = _log(rng, 1, min(65536, (1 << 26) // cols))
        return dict(op=op, fmt=fmt, rows=rows, cols=cols, stride=cols + rng.choice((0, 0, 3, 8)),
                    per_global=rng.choice((0, _log(rng, 1, rows))) if fmt == E2M1 else 0,
                    dtype=rng.choice(("float32", "bfloat16")))
    swiglu = rng.random() < 0.5
    pool = _log(rng, 1, 256)
    K = rng.randint(1, min(8, pool))
    k = 32 * _log(rng, 1, 128)
    n = _log(rng, 16, min(4096, (1 << 30) // (pool * k)))
    n += n % 2 if swiglu else 0
    T = _log(rng, 1, max(1, min(8192, (1 << 36) // (K * n * k))))
    return dict(op=op, T=T, K=K, pool=pool, n=n, k=k, swiglu=swiglu, out=rng.choice(("bfloat16", "float32")),
                skip=rng.choice((0.0, 0.1)))


def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "float32" else 2
        return {"bytes": c["T"] * (c["E"] * size + c["K"] * 8) + (c["E"] * 4 if c["bias"] else 0),
                "flops": c["T"] * c["E"] * 8}
    if c["op"] == "rows":
        n, size = c["rows"] * c["cols"], 4 if c["dtype"] == "float32" else 2
        code = n // 2 + n // (32 if c["fmt"] == MXFP4 else 16)
        return {"bytes": 2 * (n * size + code), "flops": 4 * n}
    R = c["T"] * c["K"]
    touched = c["pool"] * (1 - (1 - 1 / c["pool"]) ** R) if c["pool"] > R else c["pool"]
    if c["T"] == 1:
        touched = min(c["K"], c["pool"])
    cols = c["n"] // 2 if c["swiglu"] else c["n"]
    return {"bytes": touched * c["n"] * c["k"] * 17 / 32 + c["T"] * c["k"] * 2 + R * 4
            + R * cols * (4 if c["out"] == "float32" else 2),
            "flops": 2 * R * c["n"] * c["k"] * (1 - c["skip"])}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "route":
        T, E, K = c["T"], c["E"], c["K"]
        # N(0, 1) router logits with a popularity rank bias
        rank = torch.randperm(E, generator=g, device="cuda").float()
        logits = _randn(g, T, E) * 1.5 - 0.8 * torch.log(rank + 1)
        if c["masked"]:
            logits[torch.rand((T, E), generator=g, device="cuda") < 0.05] = -math.inf
            logits[::13] = -math.inf
        s = dict(c, logits=logits.to(getattr(torch, c["dtype"])).contiguous(),
                 bias=_randn(g, E) * 0.05 if c["bias"] else None,
                 ids=torch.empty((T, K), dtype=torch.int32, device="cuda"),
                 w=torch.empty((T, K), dtype=torch.float32, device="cuda"))
        if own:
            import expert_slot_cache_moe_amd as m
            s["router"] = m.make_router(
                score=m.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else m.MOE_SCORE_SOFTMAX,
                num_groups=c["groups"], top_groups=c["top_groups"],
                group_score=m.MOE_GROUP_TOP2 if c["group_top2"] else m.MOE_GROUP_MAX,
                renormalize=c["renorm"], scale=c["scale"], bias=s["bias"])
        return s
    if c["op"] == "rows":
        R, C = c["rows"], c["cols"]
        dt = getattr(torch, c["dtype"])
        buf = (_randn(g, R, c["stride"]) * 0.02).to(dt)
        glob = None
        if c["per_global"]:
            n = -(-R // c["per_global"])
            # amax / (6 * 448) of N(0, 0.02) rows, a little different for each matrix
            glob = 0.1 / 2688 * (0.75 + 0.5 * torch.rand(n, generator=g, device="cuda"))
        blk = 32 if c["fmt"] == MXFP4 else 16
        return dict(c, src=buf[:, :C], glob=glob,
                    codes=torch.empty((R, C // 2), dtype=torch.uint8, device="cuda"),
                    scales=torch.empty((R, C // blk), dtype=torch.uint8, device="cuda"),
                    back=torch.empty((R, C), dtype=dt, device="cuda"))
    T, K, P, n, k = c["T"], c["K"], c["pool"], c["n"], c["k"]
    # weights: quantised N(0, 0.02) rows, every matrix row drawn from 4096 of them
    base = _randn(g, 4096, k) * 0.02
    codes, scales = _pack(*_quantize_plain(base, MXFP4, None, 0)[:2])
    pick = torch.randint(0, 4096, (P * n,), generator=g, device="cuda")
    x = _randn(g, T, k).to(torch.bfloat16)
    # distinct rows for each token, popular ones more often
    pop = -0.5 * torch.log(torch.randperm(P, generator=g, device="cuda").float() + 1)
    u = torch.rand((T, P), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    idx = torch.sort(pop - torch.log(-torch.log(u)), dim=1, descending=True, stable=True)[1][:, :K].to(torch.int32)
    if c["skip"]:
        idx = torch.where(torch.rand((T, K), generator=g, device="cuda") < c["skip"], -1, idx)
    cols = n // 2 if c["swiglu"] else n
    s = dict(c, x=x, idx=idx.contiguous(), codes=codes[pick].view(P, n, k // 2),
             scales=scales[pick].view(P, n, k // 32),
             y=torch.empty((T * K, cols), dtype=getattr(torch, c["out"]), device="cuda"))
    if own:
        import expert_slot_cache_moe_amd as m
        s["bank"] = m.make_mx_bank(s["codes"], s["scales"])
        s["ws"] = torch.empty(max(m.moe_mx_product_workspace_bytes(P, n, k, T, K), 1), dtype=torch.uint8,
                              device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _route_plain(c):
    x = c["logits"].double()
    T, E = x.shape
    K, G = c["K"], c["groups"]
    ok = x > -math.inf                                            # false for NaN too
    x = torch.where(ok, x, -math.inf)
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        e = torch.where(ok, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0)
        s = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    # without a bias the scores are ordered as the logits are
    key = torch.where(ok, s + c["bias"].double(), -math.inf) if c["bias"] is not None else x
    if G > 1:
        per = torch.where(ok, s, -math.inf) if c["bias"] is None and c["group_top2"] else key
        per = per.view(T, G, E // G)
        if c["group_top2"] and E // G > 1:
            best = torch.sort(per, dim=2, descending=True, stable=True)[0]
            value = best[:, :, 0] + torch.where(best[:, :, 1] > -math.inf, best[:, :, 1], 0.0)
        else:
            value = per.amax(2)
        order = torch.sort(value, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, order, True)
        key = torch.where(kept[:, :, None], key.view(T, G, E // G), -math.inf).view(T, E)
    val, ids = torch.sort(key, dim=1, descending=True, stable=True)
    val, ids = val[:, :K], ids[:, :K]
    there = val > -math.inf
    w = torch.where(there, torch.gather(s, 1, ids), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        even = there.double() / there.sum(1, keepdim=True).clamp_min(1)
        w = torch.where(total > 0, w / total.clamp_min(1e-300), even)
    return torch.where(there, ids, -1).to(torch.int32), (w * c["scale"]).float()


def _e4m3_round(v):
    """v >= 0 (float64) to the nearest E4M3 value, ties to even, at most 448."""
    e = torch.floor(torch.log2(v.clamp_min(2.0 ** -40))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp_max(448.0)        # torch.round: ties to even


def _quantize_plain(x, fmt, glob, per_global):
    """Rows to (signed E2M1 values as magnitudes' code with a sign bit, scale codes, values)."""
    R, C = x.shape
    blk = 32 if fmt == MXFP4 else 16
    b = x.reshape(R, C // blk, blk)
    amax = b.abs().amax(2).double()
    if fmt == MXFP4:
        e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 125)
        scale = torch.ldexp(torch.ones_like(amax), e)
        sc = (e + 127).to(torch.uint8)
        unit = scale
    else:
        g = torch.ones((R, 1), dtype=torch.float64, device=x.device) if glob is None else \
            glob.double()[torch.arange(R, device=x.device) // per_global][:, None]
        scale = _e4m3_round(amax / (6 * g))
        sc = scale.float().to(torch.float8_e4m3fn).view(torch.uint8)
        unit = scale * g
    m = b.abs()
    code = torch.zeros(b.shape, dtype=torch.uint8, device=x.device)
    u = unit[:, :, None]
    code += m > 0.25 * u
    code += m >= 0.75 * u
    code += m > 1.25 * u
    code += m >= 1.75 * u
    code += m > 2.5 * u
    code += m >= 3.5 * u
    code += m > 5.0 * u
    code = torch.where(u > 0, code, 0) | (torch.signbit(b).to(torch.uint8) << 3)
    return code.reshape(R, C), sc, unit


def _pack(code, scales):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), scales


def _signed_values(device):
    v = torch.tensor(E2M1_VALUES, dtype=torch.float32, device=device)
    return torch.cat((v, -v))


def _rows_plain(c):
    x = c["src"]
    code, sc, unit = _quantize_plain(x, c["fmt"], c["glob"], c["per_global"])
    code, _ = _pack(code, sc)
    pair = _byte_values(x.device)
    blk = 32 if c["fmt"] == MXFP4 else 16
    v = pair[code.int()].view(x.shape[0], x.shape[1] // blk, blk)
    return (v * unit[:, :, None]).view(x.shape).to(c["back"].dtype)


def _byte_values(device):
    v = _signed_values(device)
    b = torch.arange(256, device=device)
    return torch.stack((v[b & 15], v[b >> 4]), 1)


def _product_plain(c):
    T, K, n, k = c["T"], c["K"], c["n"], c["k"]
    code, _, unit = _quantize_plain(c["x"], MXFP4, None, 0)
    q = (_signed_values(code.device)[code.int()].view(T, k // 32, 32) * unit[:, :, None].float()).view(T, k)
    # the routes of each matrix side by side, padded to the longest list
    row = c["idx"].reshape(-1).long()
    live = (row >= 0) & (row < c["pool"])
    row, route = row[live], torch.nonzero(live)[:, 0]
    by = torch.sort(row, stable=True)[1]
    row, route = row[by], route[by]
    mats, at, count = torch.unique_consecutive(row, return_inverse=True, return_counts=True)
    place = torch.arange(row.numel(), device=row.device) - (torch.cumsum(count, 0) - count)[at]
    most = int(count.max()) if row.numel() else 1
    a = torch.zeros((mats.numel(), most, k), dtype=torch.float32, device=row.device)
    a[at, place] = q[route // K]
    w = _byte_values(row.device)[c["codes"][mats].int()].view(-1, n, k // 32, 32)
    w.mul_(torch.exp2(c["scales"][mats].float() - 127)[..., None])
    y = torch.bmm(a, w.view(-1, n, k).transpose(1, 2).contiguous())
    out = torch.zeros((T * K, n), dtype=torch.float32, device=row.device)
    out[route] = y[at, place]
    if c["swiglu"]:
        gate, up = out[:, :n // 2], out[:, n // 2:]
        out = gate / (1 + torch.exp(-gate)) * up
    return out.to(c["y"].dtype)


def run(state):
    c = state
    if not own:
        return {"route": _route_plain, "rows": _rows_plain, "product": _product_plain}[c["op"]](c)
    import expert_slot_cache_moe_amd as m
    if c["op"] == "route":
        m.moe_route(c["router"], c["logits"], c["K"], c["ids"], c["w"])
        return c["ids"], c["w"]
    if c["op"] == "rows":
        fmt = m.MOE_FMT_MXFP4 if c["fmt"] == MXFP4 else m.MOE_FMT_E2M1
        m.moe_quantize_rows(fmt, c["src"], c["codes"], c["scales"], globals=c["glob"],
                            rows_per_global=c["per_global"])
        m.moe_dequantize_rows(fmt, c["codes"], c["scales"], c["back"], globals=c["glob"],
                              rows_per_global=c["per_global"])
        return c["back"]
    m.moe_mx_product(c["bank"], c["x"], c["idx"], c["y"], c["ws"], swiglu=c["swiglu"])
    return c["y"]


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_route(s):
    x = s["logits"].double().cpu().numpy()
    T, E = x.shape
    K, G = s["K"], s["groups"]
    ok = ~np.isnan(x) & (x != -np.inf)
    xm = np.where(ok, x, -np.inf)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if s["score"] == "sigmoid":
            sc = np.where(ok, 1.0 / (1.0 + np.exp(-xm)), 0.0)
        else:
            top = np.max(xm, axis=1, keepdims=True)
            ex = np.where(ok, np.exp(xm - np.where(np.isfinite(top), top, 0.0)), 0.0)
            z = ex.sum(1, keepdims=True)
            sc = np.where(z > 0, ex / np.where(z > 0, z, 1.0), 0.0)
    with_bias = s["bias"] is not None
    key = np.where(ok, sc + s["bias"].double().cpu().numpy(), -np.inf) if with_bias else xm
    if G > 1:
        src = np.where(ok, sc, -np.inf) if (s["group_top2"] and not with_bias) else key
        ordered = -np.sort(-src.reshape(T, G, E // G), axis=2)
        value = ordered[:, :, 0]
        if s["group_top2"] and E // G > 1:
            second = ordered[:, :, 1]
            value = value + np.where(second > -np.inf, second, 0.0)
        rank = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1, kind="stable")
        keep = np.repeat(rank < s["top_groups"], E // G, axis=1)
        key = np.where(keep, key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :K]
    there = np.take_along_axis(key, ids, 1) > -np.inf
    w = np.where(there, np.take_along_axis(sc, ids, 1), 0.0)
    if s["renorm"]:
        tot = w.sum(1, keepdims=True)
        even = there / np.maximum(there.sum(1, keepdims=True), 1)
        w = np.where(tot > 0, w / np.where(tot > 0, tot, 1.0), even)
    return np.where(there, ids, -1).astype(np.int32), w * s["scale"]


def _exact_blocks(x, fmt, glob):
    """x float64 [blocks, B], glob float64 [blocks, 1]: the values the 4-bit blocks stand for."""
    v = torch.tensor(E2M1_VALUES, dtype=torch.float64, device=x.device)
    amax = x.abs().max(1, keepdim=True).values
    if fmt == MXFP4:
        unit = torch.exp2(torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0))) - 2)
        unit = torch.where(amax > 0, unit, 1.0)
    else:
        t = amax / (6 * glob)
        table = torch.arange(127, device=x.device)
        e, mant = table // 8, (table % 8).double()
        grid = torch.where(e == 0, mant * 2.0 ** -9, (1 + mant / 8) * torch.exp2(e.double() - 7))
        hi = torch.searchsorted(grid, t.contiguous()).clamp(1, 126)
        lo = hi - 1
        down, up = t - grid[lo], grid[hi] - t
        pick = torch.where(down < up, lo, torch.where(up < down, hi, torch.where(lo % 2 == 0, lo, hi)))
        unit = grid[pick] * glob
    y = x.abs() / torch.where(unit > 0, unit, 1.0)
    hi = torch.searchsorted(v, y.contiguous()).clamp(1, 7)
    lo = hi - 1
    # distances to the neighbours in units of the scale, exactly: |x| - v * unit
    down, up = x.abs() - v[lo] * unit, v[hi] * unit - x.abs()
    pick = torch.where(down < up, lo, torch.where(up < down, hi, torch.where(lo % 2 == 0, lo, hi)))
    return torch.where(unit > 0, v[pick] * unit, 0.0) * torch.where(torch.signbit(x), -1.0, 1.0)


def _exact_quantized(x, fmt, glob, per_global):
    R, C = x.shape
    B = 32 if fmt == MXFP4 else 16
    g = torch.ones(R, dtype=torch.float64, device=x.device) if glob is None else \
        torch.repeat_interleave(glob.double(), per_global)[:R]
    out = torch.empty((R, C), dtype=torch.float64, device=x.device)
    for r in range(0, R, 4096):
        part = x[r:r + 4096].double().reshape(-1, B)
        gg = torch.repeat_interleave(g[r:r + 4096], C // B)[:, None]
        out[r:r + 4096] = _exact_blocks(part, fmt, gg).view(-1, C)
    return out


def _exact_product(s):
    T, K, n, k = s["T"], s["K"], s["n"], s["k"]
    q = _exact_quantized(s["x"], MXFP4, None, 0)
    vals = torch.tensor(E2M1_VALUES + tuple(-v for v in E2M1_VALUES), dtype=torch.float64, device=q.device)
    out = torch.zeros((T * K, n), dtype=torch.float64, device=q.device)
    rows = s["idx"].reshape(-1)
    for p in range(s["pool"]):
        route = torch.nonzero(rows == p)[:, 0]
        if not route.numel():
            continue
        b = s["codes"][p].long()
        w = torch.stack((vals[b & 15], vals[b >> 4]), 2).view(n, k // 32, 32)
        w = (w * torch.exp2(s["scales"][p].double() - 127)[:, :, None]).view(n, k)
        out[route] = q[route // K] @ w.t().contiguous()
    if s["swiglu"]:
        gate, up = out[:, :n // 2], out[:, n // 2:]
        out = gate * torch.sigmoid(gate) * up
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "rows":
        return _exact_quantized(s["src"], s["fmt"], s["glob"], s["per_global"])
    return _exact_product(s)
