"""Timing cases of the lists of routes by expert, the ragged products grouped
by expert, and the dense product with bias, activation and residual.

With `own` false, run() computes each operator in plain torch operations
(32-bit floats); with `own` true it makes the library calls a serving program
makes.  exact() is the definition in 64 bits.

  lists    routes [T, K] sorted by the matrix they name, and where each
           matrix's routes begin
  grouped  rows that lie side by side by matrix, each times its matrix: bf16,
           E2M1 or MXFP4 weights, bf16 rows; rows gathered from the tokens
           or results scattered to the routes
  linear   every row times one matrix, plus bias, activation and residual
"""
import math

import numpy as np
import torch

own = False

BF16, E2M1, MXFP4 = "bf16", "e2m1", "mxfp4"
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token's 8 experts of 256
        dict(name="lists-token", op="lists", T=1, K=8, P=256, skip=0.0),
        # a long prompt over 512 experts, top 10, some routes without a row
        dict(name="lists-prompt", op="lists", T=16384, K=10, P=512, skip=0.02),
        # one token's gate/up over its 8 experts (256 experts, H 2048, F 512)
        dict(name="grouped-token", op="grouped", fmt=BF16, T=1, K=8, P=256, n=1024, k=2048, way="gather",
             act="swiglu", bias=False, out="bfloat16", skip=0.0, pad=0),
        # the wide decode step's gate/up: 600 rows, top 2 of 160 experts, H 1024, F 256
        dict(name="grouped-wide", op="grouped", fmt=E2M1, T=600, K=2, P=160, n=512, k=1024, way="gather",
             act="swiglu", bias=False, out="bfloat16", skip=0.0, pad=0),
        # odd sizes, rows cut out of a wider buffer, a bias, some matrices not there
        dict(name="grouped-odd", op="grouped", fmt=BF16, T=45, K=3, P=24, n=515, k=1061, way="rows",
             act="none", bias=True, out="float32", skip=0.1, pad=6),
        # a short prompt's gate/up over the 256 experts of the 4096-wide layer, about 24 rows each
        dict(name="grouped-short", op="grouped", fmt=E2M1, T=1024, K=6, P=256, n=2048, k=4096, way="gather",
             act="swiglu", bias=False, out="bfloat16", skip=0.0, pad=0),
        # a prompt's gate/up over the same layer (F 1024)
        dict(name="grouped-prompt", op="grouped", fmt=BF16, T=4096, K=6, P=256, n=2048, k=4096, way="gather",
             act="swiglu", bias=False, out="bfloat16", skip=0.0, pad=0),
        # its down projection from an MXFP4 bank, fp32 rows in the routes' order
        dict(name="grouped-prompt-down", op="grouped", fmt=MXFP4, T=4096, K=6, P=256, n=4096, k=1024,
             way="scatter", act="none", bias=False, out="float32", skip=0.0, pad=0),
        # one token's router logits (256 experts, H 2048)
        dict(name="linear-router", op="linear", T=1, n=256, k=2048, act="none", bias=True, residual=False,
             out="float32", pad=0),
        # a dense down projection of the wide step's rows, added to the residual stream
        dict(name="linear-batch", op="linear", T=600, n=1024, k=256, act="none", bias=False, residual=True,
             out="bfloat16", pad=0),
        # odd sizes, rows cut out of a wider buffer
        dict(name="linear-odd", op="linear", T=77, n=515, k=1061, act="gelu", bias=True, residual=True,
             out="bfloat16", pad=6),
        # a dense layer over a long prompt
        dict(name="linear-prompt", op="linear", T=8192, n=4096, k=4096, act="silu", bias=True, residual=True,
             out="bfloat16", pad=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("lists", "grouped", "grouped", "linear"))
    if op == "lists":
        P = _log(rng, 1, 512)
        K = rng.randint(1, min(16, P))
        return dict(op=op, T=_log(rng, 1, 163840 // K), K=K, P=P, skip=rng.choice((0.0, 0.02, 0.3)))
    act = rng.choice(("none", "silu", "gelu", "swiglu"))
    out = rng.choice(("bfloat16", "float32"))
    if op == "linear":
        k = _log(rng, 1, 4096) if rng.random() < 0.4 else 8 * _log(rng, 1, 512)
        n = _log(rng, 2, 4096)
        n += n % 2 if act == "swiglu" else 0
        return dict(op=op, T=_log(rng, 1, 8192), n=n, k=k, act=act, bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, out=out, pad=rng.choice((0, 0, 3, 8)))
    fmt = rng.choice((BF16, E2M1, MXFP4))
    P = _log(rng, 1, 256)
    K = rng.randint(1, min(8, P))
    k = 32 * _log(rng, 1, 128) if fmt != BF16 or rng.random() < 0.6 else _log(rng, 1, 4096)
    n = _log(rng, 2, min(4096, (1 << 30) // (P * k)))
    n += n % 2 if act == "swiglu" else 0
    T = _log(rng, 1, max(1, min(8192, (1 << 36) // (K * n * k))))
    return dict(op=op, fmt=fmt, T=T, K=K, P=P, n=n, k=k, way=rng.choice(("gather", "rows", "scatter")), act=act,
                bias=rng.random() < 0.3, out=out, skip=rng.choice((0.0, 0.1)), pad=rng.choice((0, 0, 3, 8)))


def _cols(c):
    return c["n"] // 2 if c["act"] == "swiglu" else c["n"]


def work(case):
    c = case
    if c["op"] == "lists":
        return {"bytes": c["T"] * c["K"] * 8 + (c["P"] + 1) * 4, "flops": c["T"] * c["K"]}
    size = 4 if c["out"] == "float32" else 2
    if c["op"] == "linear":
        return {"bytes": 2 * c["n"] * c["k"] + c["T"] * (2 * c["k"] + _cols(c) * (size + 2 * c["residual"]))
                + 4 * c["n"] * c["bias"],
                "flops": 2 * c["T"] * c["n"] * c["k"]}
    R, P = c["T"] * c["K"], c["P"]
    live = R * (1 - c["skip"])
    touched = min(c["K"], P) if c["T"] == 1 else P * (1 - (1 - 1 / P) ** live) if P > 1 else 1
    weight = {BF16: 2, E2M1: 9 / 16, MXFP4: 17 / 32}[c["fmt"]]
    rows = c["T"] if c["way"] == "gather" else live
    return {"bytes": touched * c["n"] * (c["k"] * weight + 4 * c["bias"]) + rows * c["k"] * 2 + live * _cols(c) * size
            + (P + 1) * 4 + (0 if c["way"] == "rows" else R * 4),
            "flops": 2 * live * c["n"] * c["k"]}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _routes(c, g):
    """Distinct rows for each token, popular ones more often; some routes without a row."""
    T, K, P = c["T"], c["K"], c["P"]
    pop = -0.5 * torch.log(torch.randperm(P, generator=g, device="cuda").float() + 1)
    u = torch.rand((T, P), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    idx = torch.sort(pop - torch.log(-torch.log(u)), dim=1, descending=True, stable=True)[1][:, :K].to(torch.int32)
    if c["skip"]:
        idx = torch.where(torch.rand((T, K), generator=g, device="cuda") < c["skip"], -1, idx)
    return idx.contiguous()


def _lists(idx, P):
    """Route numbers sorted by row, those without one last, and the first place of each row."""
    row = idx.reshape(-1).long()
    row = torch.where((row >= 0) & (row < P), row, P)
    row, order = torch.sort(row, stable=True)
    offsets = torch.searchsorted(row, torch.arange(P + 1, device=row.device))
    return offsets.to(torch.int32), order.to(torch.int32)


def _quantized(x, fmt):
    """Rows of weights to codes, scales and, for E2M1, one global scale."""
    R, C = x.shape
    blk = 32 if fmt == MXFP4 else 16
    b = x.view(R, C // blk, blk)
    amax = b.abs().amax(2).clamp_min(1e-20)
    if fmt == MXFP4:
        e = torch.floor(torch.log2(amax)) - 2
        unit, scales, glob = torch.exp2(e), (e + 127).to(torch.uint8), None
    else:
        glob = float(amax.max()) / (6 * 448)
        s = (amax / (6 * glob)).to(torch.float8_e4m3fn)
        unit, scales = s.float() * glob, s.view(torch.uint8)
    mids = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=x.device)
    code = torch.bucketize((b.abs() / unit.clamp_min(1e-30)[:, :, None]).contiguous(), mids).to(torch.uint8)
    code = (code | (torch.signbit(b).to(torch.uint8) << 3)).view(R, C)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), scales, glob


def _rows(g, rows, k, pad):
    """bf16 rows, cut out of a wider buffer where pad is not 0."""
    return _randn(g, rows, k + pad).to(torch.bfloat16)[:, :k]


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "lists":
        T, K, P = c["T"], c["K"], c["P"]
        s = dict(c, idx=_routes(c, g), offsets=torch.empty(P + 1, dtype=torch.int32, device="cuda"),
                 order=torch.empty(T * K, dtype=torch.int32, device="cuda"))
        if own:
            import expert_slot_cache_moe_amd as m
            s["ws"] = torch.empty(max(m.moe_group_routes_workspace_bytes(P, T, K), 1), dtype=torch.uint8,
                                  device="cuda")
        return s
    n, k, out = c["n"], c["k"], getattr(torch, c["out"])
    if c["op"] == "linear":
        s = dict(c, x=_rows(g, c["T"], k, c["pad"]), w=(_randn(g, n, k) * 0.02).to(torch.bfloat16),
                 b=_randn(g, n) * 0.1 if c["bias"] else None,
                 res=_randn(g, c["T"], _cols(c)).to(torch.bfloat16) if c["residual"] else None,
                 y=torch.empty((c["T"], _cols(c)), dtype=out, device="cuda"))
        if own:
            import expert_slot_cache_moe_amd as m
            s["bank"] = m.make_bank(m.MOE_FMT_BF16, s["w"].view(1, n, k))
        return s
    T, K, P, fmt = c["T"], c["K"], c["P"], c["fmt"]
    idx = _routes(c, g)
    offsets, order = _lists(idx, P)
    base = _randn(g, 4096, k) * 0.02
    pick = torch.randint(0, 4096, (P * n,), generator=g, device="cuda")
    s = dict(c, scales=None, glob=None)
    if fmt == BF16:
        s["w"] = base.to(torch.bfloat16)[pick].view(P, n, k)
    else:
        codes, scales, glob = _quantized(base, fmt)
        s["w"], s["scales"] = codes[pick].view(P, n, k // 2), scales[pick].view(P, n, -1)
        if glob is not None:
            # a little different for each matrix
            s["glob"] = glob * (0.75 + 0.5 * torch.rand(P, generator=g, device="cuda"))
    s.update(offsets=offsets, order=order, mats=None, b=_randn(g, P, n) * 0.1 if c["bias"] else None,
             x=_rows(g, T if c["way"] == "gather" else T * K, k, c["pad"]),
             y=torch.zeros((T * K, _cols(c)), dtype=out, device="cuda"))
    if c["way"] == "rows":
        # the groups' matrices in another order, some of them not there
        s["mats"] = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        if c["skip"]:
            s["mats"] = torch.where(torch.rand(P, generator=g, device="cuda") < c["skip"], -1, s["mats"])
    if own:
        import expert_slot_cache_moe_amd as m
        f = {BF16: m.MOE_FMT_BF16, E2M1: m.MOE_FMT_E2M1, MXFP4: m.MOE_FMT_MXFP4}[fmt]
        s["bank"] = m.make_bank(f, s["w"], s["scales"], s["glob"])
    return s


# ---------------------------------------------------------------- plain forms

def _act_plain(y, act):
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "swiglu":
        gate, up = y[:, :y.shape[1] // 2], y[:, y.shape[1] // 2:]
        return gate / (1 + torch.exp(-gate)) * up
    return y


def _weights_plain(c, mats):
    """The matrices `mats` in 32 bits."""
    if c["fmt"] == BF16:
        return c["w"][mats].float()
    v = torch.tensor(E2M1_VALUES + tuple(-v for v in E2M1_VALUES), dtype=torch.float32, device=mats.device)
    b = torch.arange(256, device=mats.device)
    pair = torch.stack((v[b & 15], v[b >> 4]), 1)
    blk = 32 if c["fmt"] == MXFP4 else 16
    w = pair[c["w"][mats].int()].view(mats.numel(), c["n"], c["k"] // blk, blk)
    s = c["scales"][mats]
    if c["fmt"] == MXFP4:
        w.mul_(torch.exp2(s.float() - 127)[..., None])
    else:
        w.mul_((s.view(torch.float8_e4m3fn).float() * c["glob"][mats][:, None, None])[..., None])
    return w.view(mats.numel(), c["n"], c["k"])


def _grouped_plain(c):
    R, n, k, P = c["T"] * c["K"], c["n"], c["k"], c["P"]
    off = c["offsets"].long()
    place = torch.arange(R, device=off.device)
    group = torch.searchsorted(off, place, right=True) - 1       # P past the last group
    mat = torch.where(group < P, (c["mats"].long() if c["mats"] is not None else
                                  torch.arange(P, device=off.device))[group.clamp_max(P - 1)], -1)
    # the places of each matrix side by side, padded to the longest list
    place = place[mat >= 0]
    mat, group = mat[place], group[place]
    used, at, count = torch.unique_consecutive(group, return_inverse=True, return_counts=True)
    out = torch.zeros((R, _cols(c)), dtype=c["y"].dtype, device=off.device)
    if not place.numel():
        return out
    mats = mat[torch.cumsum(count, 0) - 1]
    most = int(count.max())
    step = max(1, (1 << 31) // (n * k))                           # so many matrices at a time
    first = torch.cumsum(count, 0) - count
    for i in range(0, used.numel(), step):
        rows = torch.nonzero((at >= i) & (at < i + step))[:, 0]
        a = torch.zeros((min(step, used.numel() - i), most, k), dtype=torch.float32, device=off.device)
        src = place[rows]
        if c["way"] == "gather":
            src = c["order"].long()[src] // c["K"]
        a[at[rows] - i, rows - first[at[rows]]] = c["x"][src].float()
        w = _weights_plain(c, mats[i:i + step]).transpose(1, 2).contiguous()
        y = torch.bmm(a, w)[at[rows] - i, rows - first[at[rows]]]
        if c["b"] is not None:
            y = y + c["b"][mat[rows]]
        dst = place[rows]
        if c["way"] == "scatter":
            dst = c["order"].long()[dst]
        out[dst] = _act_plain(y, c["act"]).to(out.dtype)
    return out


def _linear_plain(c):
    y = c["x"].float() @ c["w"].float().t()
    if c["b"] is not None:
        y = y + c["b"]
    y = _act_plain(y, c["act"])
    if c["res"] is not None:
        y = y + c["res"].float()
    return y.to(c["y"].dtype)


def run(state):
    c = state
    if not own:
        if c["op"] == "lists":
            return _lists(c["idx"], c["P"])
        return _grouped_plain(c) if c["op"] == "grouped" else _linear_plain(c)
    import expert_slot_cache_moe_amd as m
    if c["op"] == "lists":
        m.moe_group_routes(c["idx"], c["P"], c["offsets"], c["order"], c["ws"])
        return c["offsets"], c["order"]
    act = {"none": m.MOE_ACT_NONE, "silu": m.MOE_ACT_SILU, "gelu": m.MOE_ACT_GELU,
           "swiglu": m.MOE_ACT_SWIGLU}[c["act"]]
    if c["op"] == "linear":
        m.moe_linear(c["bank"], c["x"], c["y"], activation=act, bias=c["b"], residual=c["res"])
        return c["y"]
    gather = c["way"] == "gather"
    m.moe_grouped_product(c["bank"], c["x"], c["offsets"], c["y"], matrices=c["mats"],
                          gather=c["order"] if gather else None, gather_div=c["K"] if gather else 1,
                          scatter=c["order"] if c["way"] == "scatter" else None, activation=act, bias=c["b"])
    return c["y"]


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_lists(s):
    row = s["idx"].cpu().numpy().reshape(-1)
    row = np.where((row < 0) | (row >= s["P"]), s["P"], row)
    count = np.bincount(row, minlength=s["P"] + 1)[:s["P"]]
    return (np.concatenate(([0], np.cumsum(count))).astype(np.int32),
            np.argsort(row, kind="stable").astype(np.int32))


def _exact_act(y, act):
    if act == "silu":
        return y * torch.sigmoid(y)
    if act == "gelu":
        return y * 0.5 * torch.special.erfc(-y / math.sqrt(2.0))
    if act == "swiglu":
        gate, up = y.chunk(2, dim=1)
        return gate * torch.sigmoid(gate) * up
    return y


def _exact_matrix(s, p):
    if s["fmt"] == BF16:
        return s["w"][p].double()
    b = s["w"][p].long()
    vals = torch.tensor(E2M1_VALUES + tuple(-v for v in E2M1_VALUES), dtype=torch.float64, device=b.device)
    w = torch.stack((vals[b & 15], vals[b >> 4]), 2).view(s["n"], s["k"])
    sc = s["scales"][p]
    if s["fmt"] == MXFP4:
        unit = torch.exp2(sc.double() - 127)
    else:
        e, mant = (sc >> 3).double(), (sc & 7).double()
        unit = torch.where(e > 0, (1 + mant / 8) * torch.exp2(e - 7), mant * 2.0 ** -9) * s["glob"][p].double()
    return w * torch.repeat_interleave(unit, s["k"] // unit.shape[1], dim=1)


def _exact_grouped(s):
    y = torch.zeros((s["T"] * s["K"], _cols(s)), dtype=torch.float64, device=s["x"].device)
    off = s["offsets"].tolist()
    mats = s["mats"].tolist() if s["mats"] is not None else list(range(s["P"]))
    for gi in range(s["P"]):
        if off[gi] == off[gi + 1] or mats[gi] < 0:
            continue
        at = torch.arange(off[gi], off[gi + 1], device=y.device)
        routes = s["order"].long()[at]
        x = s["x"][routes // s["K"] if s["way"] == "gather" else at].double()
        v = x @ _exact_matrix(s, mats[gi]).t()
        if s["b"] is not None:
            v = v + s["b"][mats[gi]].double()
        y[routes if s["way"] == "scatter" else at] = _exact_act(v, s["act"])
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lists":
        return _exact_lists(s)
    if case["op"] == "grouped":
        return _exact_grouped(s)
    v = s["x"].double() @ s["w"].double().t()
    if s["b"] is not None:
        v = v + s["b"].double()
    v = _exact_act(v, s["act"])
    return v if s["res"] is None else v + s["res"].double()
