"""The scored router, the 4-bit rows and the MXFP4 products on the GPU
against plain 64-bit forms (operator_ref.py).

Tolerances, from the arithmetic:
  - ids, codes and scales are equal; dequantized values are exact, or one
    rounding of the exact value (half a step: fp32 2^-24, bf16 2^-8);
  - routing weights: 64-bit arithmetic rounded once to fp32, 2^-24, plus the
    difference of two 64-bit exponentials (far below);
  - products: the terms are exact, an fp32 sum of k of them in any order is
    within k 2^-23 of the sum of their magnitudes (one rounding, or one
    truncation, each); then one rounding to the output's type."""
import numpy as np
import pytest
import torch

import expert_slot_cache_moe_amd as m
import operator_ref as ref
from expert_slot_cache_moe_amd import workloads as W

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _say(*a):
    print(*a, flush=True)


def _f64(t):
    return t.double().cpu().numpy()


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


# ---------------------------------------------------------------- routing

def _route(logits, K, bias=None, stream=None, **kw):
    T, E = logits.shape
    router = m.make_router(
        score=m.MOE_SCORE_SIGMOID if kw["score"] == "sigmoid" else m.MOE_SCORE_SOFTMAX,
        num_groups=kw.get("groups", 1), top_groups=kw.get("top_groups", 1),
        group_score=m.MOE_GROUP_TOP2 if kw.get("top2") else m.MOE_GROUP_MAX, renormalize=kw.get("renorm", True),
        scale=kw.get("scale", 1.0), bias=bias)
    ids = torch.full((T, K), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), np.nan, dtype=torch.float32, device="cuda")
    m.moe_route(router, logits, K, ids, w, stream=stream)
    return ids, w


def _check_route(logits, K, bias=None, **kw):
    ids, w = _route(logits, K, bias=bias, **kw)
    e_ids, e_w = ref.route(_f64(logits), K, bias=None if bias is None else _f64(bias), **kw)
    assert (ids.cpu().numpy() == e_ids).all()
    got = _f64(w)
    assert (np.abs(got - e_w) <= np.abs(e_w) * (2.0 ** -24 + 1e-12) + 2.0 ** -150).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K,kw", [
    (1, 256, 8, dict(score="sigmoid", groups=8, top_groups=4, top2=True, bias=True, scale=2.5)),
    (3, 256, 8, dict(score="sigmoid", groups=8, top_groups=4, top2=True)),
    (5, 1, 1, dict(score="softmax")),
    (9, 7, 7, dict(score="softmax", renorm=False)),
    (33, 64, 64, dict(score="sigmoid", renorm=False, bias=True)),
    (40, 160, 6, dict(score="softmax", groups=8, top_groups=3, renorm=False, scale=16.0)),
    (40, 160, 6, dict(score="softmax", groups=8, top_groups=3, top2=True, bias=True)),
    (17, 96, 5, dict(score="softmax", groups=3, top_groups=2, top2=True)),
    (17, 65, 4, dict(score="sigmoid", groups=13, top_groups=5, top2=True, bias=True)),
    (12, 64, 3, dict(score="sigmoid", groups=64, top_groups=2, top2=True)),
    (12, 63, 9, dict(score="sigmoid", groups=63, top_groups=7, bias=True)),
    (70, 512, 10, dict(score="sigmoid", bias=True)),
    (70, 512, 10, dict(score="softmax", bias=True, renorm=False)),
    (21, 640, 6, dict(score="softmax")),
    (6, 1000, 13, dict(score="sigmoid", groups=10, top_groups=1, bias=True)),
    (4, 2048, 64, dict(score="softmax", groups=16, top_groups=3, top2=True, bias=True)),
    (300, 33, 2, dict(score="softmax", groups=11, top_groups=11)),
    (600, 160, 2, dict(score="softmax")),
    (1500, 48, 4, dict(score="sigmoid", groups=4, top_groups=2, bias=True)),
    (4097, 48, 4, dict(score="sigmoid", groups=4, top_groups=2, bias=True)),
    (4098, 130, 12, dict(score="softmax", bias=True)),
    (4099, 20, 12, dict(score="softmax", renorm=False)),
    (4100, 200, 13, dict(score="sigmoid")),
])
def test_route_matches_the_plain_form(T, E, K, kw, dtype):
    _say("route", T, E, K, kw, dtype)
    g = W.rng(7, "route", T, E, K, sorted(kw.items()))
    kw = dict(kw)
    bias = torch.from_numpy((g.standard_normal(E) * 0.1).astype(np.float32)).cuda() if kw.pop("bias", False) else None
    x = torch.from_numpy((g.standard_normal((T, E)) * 2).astype(np.float32)).to(dtype).cuda()
    _check_route(x, K, bias=bias, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups,top2", [(1, 1, False), (4, 2, False), (4, 2, True)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_ties_masks_and_extremes(score, groups, top_groups, top2, with_bias):
    _say("route edges", score, groups, top_groups, top2, with_bias)
    E, K = 32, 12
    inf, nan, low = np.inf, np.nan, float(np.finfo(np.float32).min)
    rows = [
        np.zeros(E),                                            # every score equal: lower ids first
        np.repeat([1.0, 0.0], E // 2),
        np.full(E, -inf),                                       # nothing available
        np.full(E, nan),
        np.full(E, low),                                        # a mask of the type's lowest value
        np.where(np.arange(E) % 5 == 0, 0.5, -inf),             # fewer available than K
        np.where(np.arange(E) < 8, -inf, np.arange(E) / 8.0),   # a whole group masked
        np.where(np.arange(E) == 9, 2.0, -inf),                 # one expert left
        np.where(np.arange(E) == 9, 2.0, low),
        np.where(np.arange(E) % 2 == 0, nan, np.arange(E) / 4.0),
        np.tile([0.0, -0.0], E // 2),                           # both zeros are one value
        np.linspace(-80, 80, E),
    ]
    if score == "softmax" or not with_bias:
        rows.append(np.where(np.arange(E) % 7 == 3, inf, 1.0))  # +infinity shares the softmax
    x = torch.from_numpy(np.array(rows, np.float32)).cuda()
    bias = None
    if with_bias:
        b = np.zeros(E, np.float32)
        b[3], b[5], b[11], b[20] = -inf, nan, 0.25, -0.5        # -inf and NaN take an expert out
        bias = torch.from_numpy(b).cuda()
    for renorm in (True, False):
        _check_route(x, K, bias=bias, score=score, groups=groups, top_groups=top_groups, top2=top2,
                     renorm=renorm, scale=3.0)


def test_route_orders_scores_closer_than_an_fp32_rounding():
    # sigmoids near 1 differ by 1e-9; a bias keeps the score order in play
    E, K = 64, 16
    g = W.rng(3, "near")
    x = (20.0 + g.permutation(E) * 0.01).astype(np.float32)[None, :]
    bias = torch.zeros(E, dtype=torch.float32, device="cuda")
    assert len(np.unique((1 / (1 + np.exp(-x.astype(np.float64)))).astype(np.float32))) < K
    _check_route(torch.from_numpy(x).cuda(), K, bias=bias, score="sigmoid")
    # and equal upper halves of the 64-bit keys: bf16-close logits with tiny biases
    bias = torch.from_numpy((g.permutation(E) * 1e-9).astype(np.float32)).cuda()
    _check_route(torch.full((3, E), 0.75, device="cuda"), K, bias=bias, score="sigmoid")
    _check_route(torch.full((3, E), 0.75, device="cuda"), K, bias=bias, score="sigmoid", groups=8, top_groups=3,
                 top2=True)


@pytest.mark.parametrize("score,groups,top2,with_bias", [("sigmoid", 1, False, True), ("softmax", 1, False, False),
                                                         ("sigmoid", 8, True, True), ("softmax", 8, False, True)])
def test_many_rows_of_every_kind_side_by_side(score, groups, top2, with_bias):
    # four rows to a wave: rows with few candidates next to rows that are finished by themselves
    T, E, K = 4102, 192, 6
    g = W.rng(5, "many", score, groups)
    x = g.standard_normal((T, E)).astype(np.float32)
    x[1::7] = -np.inf
    x[2::7] = 0.5                                             # all equal
    x[3::7, 5:] = -np.inf                                     # fewer than K
    x[4::11] = np.round(x[4::11])                             # many equal
    x[5::11, :100] = np.finfo(np.float32).min
    x[6::13] = np.nan
    x[8::13, 20] = np.inf
    x[9::17] *= 1e-7
    bias = torch.from_numpy((g.standard_normal(E) * 0.05).astype(np.float32)).cuda() if with_bias else None
    for renorm in (True, False):
        _check_route(torch.from_numpy(x).cuda(), K, bias=bias, score=score, groups=groups,
                     top_groups=min(3, groups), top2=top2, renorm=renorm)


@pytest.mark.parametrize("E,groups,top_groups,top2", [(64, 1, 1, False), (256, 1, 1, False), (256, 8, 3, True),
                                                      (256, 8, 3, False), (1024, 16, 5, True)])
def test_route_under_biases_of_every_size(E, groups, top_groups, top2):
    g = W.rng(4, "biases", E, groups, top2)
    x = g.standard_normal((24, E)).astype(np.float32)
    x[1::4] = np.round(x[1::4] * 2) / 2                       # many equal scores
    x[2::4] = x[2::4, :1]
    inf, low = np.inf, np.finfo(np.float32).min
    for b in (np.zeros(E), np.where(np.arange(E) % 3 == 0, 1e6, -1e6), np.where(g.random(E) < 0.5, low, 0.0),
              np.where(g.random(E) < 0.02, inf, 0.1), g.standard_normal(E) * 1e-8, g.standard_normal(E) * 1e3,
              np.where(g.random(E) < 0.9, -inf, 0.0)):
        bias = torch.from_numpy(b.astype(np.float32)).cuda()
        for score in ("sigmoid", "softmax"):
            _check_route(torch.from_numpy(x).cuda(), 7, bias=bias, score=score, groups=groups, top_groups=top_groups,
                         top2=top2)


def test_route_of_strided_rows_leaves_the_rest_alone():
    g = W.rng(5, "strided")
    T, E, K = 37, 50, 4
    buf = torch.from_numpy(g.standard_normal((T, 61)).astype(np.float32)).cuda()
    x = buf[:, 3:3 + E]
    router = m.make_router(score=m.MOE_SCORE_SOFTMAX)
    ids = torch.full((T + 2, K), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 2, K), 7.0, dtype=torch.float32, device="cuda")
    m.moe_route(router, x, K, ids[1:T + 1], w[1:T + 1])
    e_ids, e_w = ref.route(_f64(x), K, score="softmax")
    assert (ids[1:T + 1].cpu().numpy() == e_ids).all()
    assert (ids[0] == 77).all() and (ids[-1] == 77).all() and (w[0] == 7).all() and (w[-1] == 7).all()


# ---------------------------------------------------------------- 4-bit rows

FMT = {"mxfp4": m.MOE_FMT_MXFP4, "e2m1": m.MOE_FMT_E2M1}


def _quantize(x, fmt, glob=None, per=0, stream=None):
    R, C = x.shape
    B = 32 if fmt == "mxfp4" else 16
    codes = torch.full((R, C // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, C // B), 0xCD, dtype=torch.uint8, device="cuda")
    m.moe_quantize_rows(FMT[fmt], x, codes, scales, globals=glob, rows_per_global=per, stream=stream)
    return codes, scales


def _check_rows(x, fmt, glob=None, per=0):
    """Quantizes x and back; everything equal to the plain form."""
    codes, scales = _quantize(x, fmt, glob, per)
    gl = None if glob is None else _f64(glob)
    e_codes, e_scales, e_vals = ref.quantize(_f64(x), fmt, gl, max(per, 1))
    assert (scales.cpu().numpy() == e_scales).all()
    assert (codes.cpu().numpy() == e_codes).all()
    for dt in (torch.float32, torch.bfloat16):
        back = torch.full((x.shape[0], x.shape[1] + 5), 9.0, dtype=dt, device="cuda")
        m.moe_dequantize_rows(FMT[fmt], codes, scales, back[:, :x.shape[1]], globals=glob, rows_per_global=per)
        got = _f64(back[:, :x.shape[1]])
        nan = np.isnan(e_vals)
        assert (np.isnan(got) == nan).all()
        with np.errstate(invalid="ignore"):
            assert (np.abs(got - e_vals)[~nan] <= HALF[dt] * np.abs(e_vals)[~nan] + 2.0 ** -134).all()
        assert (back[:, x.shape[1]:] == 9).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["mxfp4", "e2m1"])
@pytest.mark.parametrize("R,C,stride", [
    (1, 32, 32), (1, 2048, 2048), (3, 64, 64), (77, 96, 101), (50, 1056, 1061), (33, 128, 136), (700, 512, 512),
    (5, 4096, 4097),
])
def test_rows_match_the_plain_form(fmt, R, C, stride, dtype):
    _say("rows", fmt, R, C, stride, dtype)
    g = W.rng(11, "rows", fmt, R, C, stride, str(dtype))
    buf = torch.from_numpy((g.standard_normal((R, stride)) * 0.02).astype(np.float32)).to(dtype).cuda()
    x = buf[:, :C]
    _check_rows(x, fmt)
    if fmt == "e2m1":
        per = max(1, R // 3)
        glob = torch.from_numpy((g.random(-(-R // per)) * 1e-4 + 1e-5).astype(np.float32)).cuda()
        _check_rows(x, fmt, glob, per)


@pytest.mark.parametrize("fmt", ["mxfp4", "e2m1"])
def test_every_bf16_value_and_every_scale(fmt):
    # blocks of one value beside zeros, and beside the largest of their binade
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    bits = bits[np.isfinite(ref.bf16_f64(bits))]
    B = 32 if fmt == "mxfp4" else 16
    x = np.zeros((2, bits.size, B), np.uint16)
    x[:, :, 0] = bits
    x[1, :, 1] = (bits & 0x7F80) | 0x7F                # 1.99 x 2^e of the same binade
    x[1, :, 2] = np.minimum((bits & 0x7F80) + 0x100, 0x7F00) | 0x20
    t = torch.from_numpy(x.reshape(-1, B * 4).view(np.int16)).cuda().view(torch.bfloat16) \
        if x.size % (B * 4) == 0 else torch.from_numpy(x.reshape(-1, B).view(np.int16)).cuda().view(torch.bfloat16)
    _check_rows(t, fmt)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_e2m1_scales_beside_the_middle_of_two_scales(dtype):
    # the largest of a block: 6 g times a middle of two E4M3 values, one step of its type either way
    g = W.rng(12, "scale middles")
    grid = ref.e4m3_grid()
    mids = (grid[1:] + grid[:-1]) / 2
    globs = np.concatenate([[1.0, 0.5, 3.0], (g.random(29) + 0.5) * 2.0 ** g.integers(-30, 30, 29)]).astype(np.float32)
    step = lambda v, d: torch.nextafter(torch.from_numpy(v).to(dtype), torch.tensor(d, dtype=dtype)).double().numpy()
    x = np.zeros((len(globs), len(mids) * 3, 16))
    for i, gl in enumerate(globs):
        v = torch.from_numpy(6 * np.float64(gl) * mids).to(dtype).double().numpy()
        x[i, 0::3, 3], x[i, 1::3, 5], x[i, 2::3, 9] = v, -step(v, 0.0), step(v, np.inf)
        x[i, :, 10] = x[i, :, 3] * 0.3
    t = torch.from_numpy(x.reshape(len(globs), -1)).to(dtype).cuda()
    _check_rows(t, "e2m1", torch.from_numpy(globs).cuda(), 1)


def test_e2m1_values_beside_the_middle_of_two_codes():
    # every block: largest 6 s g, the rest a middle of two codes times s g, one fp32 step either way
    g = W.rng(13, "middles")
    R = 400
    glob = (g.random(R).astype(np.float32) + np.float32(0.5)) * np.float32(2.0) ** g.integers(-20, 20, R).astype(np.float32)
    glob[:100] = np.float32(2.0) ** g.integers(-8, 8, 100).astype(np.float32)
    s = ref.e4m3_grid()[g.integers(0x10, 0x70, R)]
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = np.zeros((R, 32), np.float32)
    for r in range(R):
        u = s[r] * np.float64(glob[r])
        x[r, 0] = x[r, 16] = np.float32(6 * u)
        v = (mids * u).astype(np.float32)
        x[r, 1:8] = v
        x[r, 8:15] = np.nextafter(v, np.float32(0))
        x[r, 17:24] = np.nextafter(v, np.float32(np.inf))
        x[r, 24:31] = -v
    _check_rows(torch.from_numpy(x).cuda(), "e2m1", torch.from_numpy(glob).cuda(), 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["mxfp4", "e2m1"])
def test_rows_of_extremes(fmt, dtype):
    C = 64
    big, tiny, sub = 3.0e38, 1.2e-38, 1e-41
    rows = np.zeros((12, C), np.float64)
    rows[0, 5] = np.inf
    rows[1, 40] = np.nan
    rows[2] = big
    rows[3, ::3] = -big
    rows[4] = tiny
    rows[5] = sub
    rows[6, 7] = sub
    rows[7] = -0.0
    rows[8, :32] = 1.0
    rows[9] = np.linspace(-1e-38, 1e-38, C)
    rows[10] = np.geomspace(1e-30, 1e30, C)
    rows[11] = -np.inf
    x = torch.from_numpy(rows.astype(np.float32)).to(dtype).cuda()
    _check_rows(x, fmt)
    if fmt == "e2m1":
        glob = torch.tensor([1e30, 1e-30, 0.0, -1.0, np.nan, np.inf, 1e-38, 1.0, 3e-5, 7.0, 1.0, 2.0],
                            dtype=torch.float32, device="cuda")
        codes, scales = _quantize(x, fmt, glob, 1)
        e_codes, e_scales, _ = ref.quantize(_f64(x), fmt, _f64(glob), 1)
        assert (scales.cpu().numpy() == e_scales).all() and (codes.cpu().numpy() == e_codes).all()


def test_dequantize_reads_every_code_and_scale():
    # all 256 code bytes under all 256 scale bytes, both formats (E4M3 also with its sign bit)
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()
    val = ref.VALUES[np.arange(16) & 7] * np.where(np.arange(16) & 8, -1.0, 1.0)
    pair = np.stack([val[np.arange(256) & 15], val[np.arange(256) >> 4]], 1).reshape(-1)
    for fmt, B in (("mxfp4", 32), ("e2m1", 16)):
        scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 512 // B).contiguous().cuda()
        out = torch.empty((256, 512), dtype=torch.float32, device="cuda")
        m.moe_dequantize_rows(FMT[fmt], codes, scales, out)
        sb = np.arange(256)
        if fmt == "mxfp4":
            s = np.where(sb == 255, np.nan, np.ldexp(1.0, sb - 127))
        else:
            s = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        with np.errstate(over="ignore"):
            want = (s[:, None] * pair[None, :]).astype(np.float32)
        assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)
        half = torch.empty((256, 512), dtype=torch.bfloat16, device="cuda")
        m.moe_dequantize_rows(FMT[fmt], codes, scales, half)
        assert np.array_equal(half.float().cpu().numpy(), torch.from_numpy(want).bfloat16().float().numpy(), equal_nan=True)


# ---------------------------------------------------------------- products

def _bank(g, P, n, k, lo=118, hi=130):
    codes = torch.from_numpy(g.integers(0, 256, (P, n, k // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(g.integers(lo, hi, (P, n, k // 32), dtype=np.uint8)).cuda()
    return m.make_mx_bank(codes, scales), codes.cpu().numpy(), scales.cpu().numpy()


def _idx(g, T, K, P, skip=0.1):
    idx = g.integers(0, P, (T, K)).astype(np.int32)
    bad = g.random((T, K)) < skip
    idx[bad] = g.choice(np.array([-1, P, -5, P + 100, 2**31 - 1, -2**31]), bad.sum())
    return idx


def _product(bank, x, idx, swiglu=False, out_dtype=torch.bfloat16, stream=None, R=None):
    """The product into the middle of a larger buffer whose ends must stay as they were."""
    T = x.shape[0]
    K = 1 if idx is None else idx.shape[1]
    cols = bank.n // 2 if swiglu else bank.n
    pad = 64
    buf = torch.full((T * K * cols + 2 * pad,), 123.0, dtype=out_dtype, device="cuda")
    out = buf[pad:pad + T * K * cols].view(T * K, cols)
    ws = torch.full((m.moe_mx_product_workspace_bytes(bank.num_rows, bank.n, bank.k, T, K) + 512,), 0xFF,
                    dtype=torch.uint8, device="cuda")
    m.moe_mx_product(bank, x, idx, out, ws[:-512], swiglu=swiglu, stream=stream)
    torch.cuda.synchronize()
    assert (buf[:pad] == 123).all() and (buf[-pad:] == 123).all() and (ws[-512:] == 0xFF).all()
    return out


def _check_product(bank, codes, scales, x, idx, swiglu, out_dtype):
    out = _product(bank, x, None if idx is None else torch.from_numpy(idx).cuda(), swiglu, out_dtype)
    T = x.shape[0]
    ix = np.zeros((T, 1), np.int32) if idx is None else idx
    xq = ref.quantize(_f64(x), "mxfp4")[2]
    want, mags = ref.product(codes, scales, xq, ix, swiglu)
    u = bank.k * 2.0 ** -23
    if swiglu:
        ag, au, gate, up = mags
        eg, eu = u * ag, u * au
        # |silu'| <= 1.1, |silu(g)| <= |g|; silu and the product in fp32: a few roundings, and the
        # exponent's argument is off by |g| 2^-24
        silu = np.abs(gate / (1 + np.exp(-np.clip(gate, -700, 700))))
        tol = 1.1 * eg * (np.abs(up) + eu) + silu * eu + np.abs(want) * (8 + np.abs(gate)) * 2.0 ** -23 + 2.0 ** -120
    else:
        tol = u * mags
    tol = tol + HALF[out_dtype] * np.abs(want) * (1 + 1e-3) + 1e-300
    got = _f64(out)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


SHAPES = [
    # T, K, P, n, k
    (1, 1, 1, 1, 32), (1, 8, 16, 64, 2048), (1, 3, 5, 15, 64), (2, 2, 3, 17, 96), (3, 1, 2, 16, 128),
    (7, 2, 4, 33, 160), (17, 1, 1, 48, 256), (33, 2, 3, 130, 512), (45, 3, 24, 515, 1056), (5, 4, 40, 260, 4096),
    (64, 8, 6, 128, 384), (130, 2, 3, 80, 1024), (300, 1, 2, 257, 544), (513, 2, 7, 96, 288),
    (40, 4, 70, 1040, 320), (30, 2, 90, 1101, 2112), (300, 8, 140, 512, 1024), (600, 4, 150, 250, 160),
    (350, 6, 400, 130, 256), (70, 2, 8, 4100, 480),
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,K,P,n,k", SHAPES)
def test_product_matches_the_plain_form(T, K, P, n, k, out_dtype):
    _say("product", T, K, P, n, k, out_dtype)
    g = W.rng(17, "product", T, K, P, n, k)
    bank, codes, scales = _bank(g, P, n, k)
    x = torch.from_numpy(W.normal_bf16(g, (T, k)).view(np.int16)).cuda().view(torch.bfloat16)
    idx = _idx(g, T, K, P)
    _check_product(bank, codes, scales, x, idx, False, out_dtype)
    if n % 2 == 0:
        _check_product(bank, codes, scales, x, idx, True, out_dtype)


@pytest.mark.parametrize("T,P,n,k", [(100, 64, 48, 320), (100, 64, 1030, 320), (100, 64, 1030, 2560), (33, 40, 70, 1024),
                                     (200, 64, 1026, 1024)])
def test_product_of_one_long_list_among_empty_ones(T, P, n, k):
    _say("one list", T, P, n, k)
    g = W.rng(18, "skew", T, P, n, k)
    bank, codes, scales = _bank(g, P, n, k)
    x = torch.from_numpy(W.normal_bf16(g, (T, k)).view(np.int16)).cuda().view(torch.bfloat16)
    idx = np.full((T, 1), P - 3, np.int32)
    idx[5:9] = -1
    idx[20] = 0
    _check_product(bank, codes, scales, x, idx, False, torch.float32)
    _check_product(bank, codes, scales, x, idx, True, torch.bfloat16)


# runs of 16 from prepared lists (the waves split k, or do not), of 64 for much matrix and few
# routes, of 128 and of 256, with scales in single bytes, dwords and vectors
@pytest.mark.parametrize("T,K,P,n,k,swiglu,out_dtype", [
    (700, 3, 200, 100, 160, False, torch.float32), (700, 3, 200, 100, 512, True, torch.bfloat16),
    (350, 6, 200, 700, 256, True, torch.float32), (350, 6, 200, 699, 160, False, torch.bfloat16),
    (4, 6, 30, 2048, 4096, True, torch.bfloat16), (1, 40, 40, 1999, 2112, False, torch.float32),
    (1150, 2, 40, 901, 352, False, torch.float32), (1150, 2, 40, 898, 384, True, torch.bfloat16),
    (1150, 2, 40, 900, 512, True, torch.float32), (1200, 2, 40, 896, 32, False, torch.bfloat16),
    (800, 1, 2, 22010, 2080, False, torch.float32), (800, 1, 2, 21904, 2176, True, torch.bfloat16),
    (800, 1, 2, 21906, 2560, True, torch.float32), (800, 1, 2, 21904, 2048, False, torch.bfloat16),
])
def test_product_of_every_run_length(T, K, P, n, k, swiglu, out_dtype):
    _say("run length", T, K, P, n, k, swiglu, out_dtype)
    g = W.rng(20, "runs", T, K, P, n, k)
    bank, codes, scales = _bank(g, P, n, k)
    x = torch.from_numpy(W.normal_bf16(g, (T, k)).view(np.int16)).cuda().view(torch.bfloat16)
    _check_product(bank, codes, scales, x, _idx(g, T, K, P, 0.02), swiglu, out_dtype)


@pytest.mark.parametrize("T,n,k", [(20, 22000, 32), (30, 16500, 416), (47, 40, 608), (50, 40, 608), (1100, 16200, 2080),
                                   (1025, 4150, 96)])
def test_dense_product_of_every_run_length(T, n, k):
    _say("dense run length", T, n, k)
    g = W.rng(21, "dense runs", T, n, k)
    bank, codes, scales = _bank(g, 1, n, k)
    x = torch.from_numpy(W.normal_bf16(g, (T, k)).view(np.int16)).cuda().view(torch.bfloat16)
    _check_product(bank, codes, scales, x, None, False, torch.float32)


@pytest.mark.parametrize("T,n,k", [(1, 70, 96), (16, 16, 128), (100, 300, 640), (257, 129, 256), (1000, 64, 2048)])
def test_dense_product_without_ids(T, n, k):
    g = W.rng(19, "dense", T, n, k)
    bank, codes, scales = _bank(g, 1, n, k)
    x = torch.from_numpy(W.normal_bf16(g, (T, k)).view(np.int16)).cuda().view(torch.bfloat16)
    _check_product(bank, codes, scales, x, None, False, torch.float32)


@pytest.mark.parametrize("T,K,P,n,k", [(4, 2, 3, 40, 32), (40, 3, 9, 100, 416), (600, 2, 4, 256, 1024), (9, 4, 8, 33, 96)])
def test_product_with_exact_sums_is_exact(T, K, P, n, k):
    # every scale a power of two shared by its row and every x block of scale 1: the terms are
    # multiples of 1/4 of at most 36, so their fp32 sums are exact in any order
    g = W.rng(23, "exact", T, K, P, n, k)
    assert k * 36 * 4 < 2 ** 24
    codes = g.integers(0, 256, (P, n, k // 2), dtype=np.uint8)
    scales = np.repeat(g.integers(100, 140, (P, n, 1), dtype=np.uint8), k // 32, axis=2)
    bank = m.make_mx_bank(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = ref.VALUES[g.integers(0, 8, (T, k))] * g.choice([-1.0, 1.0], (T, k))
    x[:, ::32] = 6.0
    xt = torch.from_numpy(x).to(torch.bfloat16).cuda()
    idx = _idx(g, T, K, P)
    out = _product(bank, xt, torch.from_numpy(idx).cuda(), out_dtype=torch.float32)
    want, _ = ref.product(codes, scales, x, idx)
    assert np.array_equal(_f64(out), want)


def test_product_reads_strided_and_unaligned_rows():
    g = W.rng(29, "strided product")
    T, K, P, n, k = 21, 2, 3, 50, 224
    bank, codes, scales = _bank(g, P, n, k)
    buf = torch.from_numpy(W.normal_bf16(g, (T, k + 13)).view(np.int16)).cuda().view(torch.bfloat16)
    for off in (0, 3, 8):
        _check_product(bank, codes, scales, buf[:, off:off + k], _idx(g, T, K, P), False, torch.float32)


def test_product_of_routes_that_all_miss_is_zero_rows():
    g = W.rng(31, "miss")
    bank, codes, scales = _bank(g, 3, 40, 64)
    for T, K in ((1, 1), (1, 4), (70, 2), (400, 1)):
        x = torch.from_numpy(W.normal_bf16(g, (T, 64)).view(np.int16)).cuda().view(torch.bfloat16)
        idx = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
        assert (_product(bank, x, idx) == 0).all()
        assert (_product(bank, x, idx, swiglu=True, out_dtype=torch.float32) == 0).all()


@pytest.mark.parametrize("T,K,P", [(1, 2, 4), (40, 2, 4), (300, 2, 2)])
def test_product_carries_nan_and_only_where_it_is_read(T, K, P):
    g = W.rng(37, "nan", T)
    n, k = 48, 256
    bank, codes, scales = _bank(g, P, n, k)
    scales[1, 5, 3] = 255
    bank = m.make_mx_bank(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = torch.from_numpy(W.normal_bf16(g, (T, k)).view(np.int16)).cuda().view(torch.bfloat16)
    if T > 3:
        x[2, 77] = float("nan")
        x[3, 200] = float("inf")
    idx = np.stack([g.permutation(P)[:K] for _ in range(T)]).astype(np.int32)
    out = _f64(_product(bank, x, torch.from_numpy(idx).cuda(), out_dtype=torch.float32))
    nan = np.zeros((T * K, n), bool)
    nan[idx.reshape(-1) == 1, 5] = True
    if T > 3:
        nan[2 * K:4 * K] = True
    assert (np.isnan(out) == nan).all()


def test_a_routes_result_depends_on_its_row_and_x_alone():
    # the same (row, x) pairs, alone, in a crowd and in another order, to the bit
    g = W.rng(41, "alone")
    P, n, k = 5, 96, 576
    bank, _, _ = _bank(g, P, n, k)
    T = 400
    x = torch.from_numpy(W.normal_bf16(g, (T, k)).view(np.int16)).cuda().view(torch.bfloat16)
    idx = torch.from_numpy(_idx(g, T, 1, P)).cuda()
    full = _product(bank, x, idx, out_dtype=torch.float32)
    again = _product(bank, x, idx, out_dtype=torch.float32)
    assert torch.equal(full, again)
    perm = torch.from_numpy(g.permutation(T)).cuda()
    assert torch.equal(_product(bank, x[perm].contiguous(), idx[perm].contiguous(), out_dtype=torch.float32), full[perm])


# ---------------------------------------------------------------- graphs, streams, arguments

def test_captured_operators_replay():
    g = W.rng(43, "graph")
    T, E, K, n, k = 24, 16, 4, 96, 288
    bank, _, _ = _bank(g, E, n, k)
    router = m.make_router(score=m.MOE_SCORE_SIGMOID, num_groups=4, top_groups=2, group_score=m.MOE_GROUP_TOP2,
                           bias=torch.from_numpy((g.standard_normal(E) * 0.1).astype(np.float32)).cuda())
    logits = torch.zeros((T, E), device="cuda")
    x = torch.zeros((T, k), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((T, K), dtype=torch.int32, device="cuda")
    w = torch.empty((T, K), device="cuda")
    y = torch.empty((T * K, n), device="cuda")
    ws = torch.empty(m.moe_mx_product_workspace_bytes(E, n, k, T, K), dtype=torch.uint8, device="cuda")
    codes = torch.empty((T, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, k // 32), dtype=torch.uint8, device="cuda")
    back = torch.empty((T, k), device="cuda")

    def step():
        m.moe_route(router, logits, K, ids, w)
        m.moe_mx_product(bank, x, ids, y, ws)
        m.moe_quantize_rows(m.MOE_FMT_MXFP4, x, codes, scales)
        m.moe_dequantize_rows(m.MOE_FMT_MXFP4, codes, scales, back)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        logits.copy_(torch.from_numpy(g.standard_normal((T, E)).astype(np.float32)))
        x.copy_(torch.from_numpy(g.standard_normal((T, k)).astype(np.float32)).to(torch.bfloat16))
        if i == 2:
            logits[::3] = -float("inf")
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (ids, w, y, codes, scales, back)]
        for t in (ids, w, y, codes, scales, back):
            t.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (ids, w, y, codes, scales, back)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,K,P,n,k", [(300, 2, 20, 130, 288), (1150, 2, 40, 900, 352), (700, 3, 200, 100, 160)])
def test_captured_product_of_prepared_lists_replays(T, K, P, n, k):
    g = W.rng(44, "graph lists", T)
    bank, _, _ = _bank(g, P, n, k)
    x = torch.zeros((T, k), dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros((T, K), dtype=torch.int32, device="cuda")
    y = torch.empty((T * K, n), device="cuda")
    ws = torch.empty(m.moe_mx_product_workspace_bytes(P, n, k, T, K), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.moe_mx_product(bank, x, idx, y, ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_mx_product(bank, x, idx, y, ws)
    for i in range(4):
        x.copy_(torch.from_numpy(g.standard_normal((T, k)).astype(np.float32)).to(torch.bfloat16))
        idx.copy_(torch.from_numpy(_idx(g, T, K, P, 0.3 * i)))
        if i == 2:
            idx[:T // 2] = 3                # half of the routes on one matrix
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.fill_(-7.0)
        m.moe_mx_product(bank, x, idx, y, ws)
        torch.cuda.synchronize()
        assert torch.equal(got, y)


def test_products_on_two_streams_at_once():
    g = W.rng(45, "two streams")
    jobs = []
    for T, K, P, n, k in ((400, 2, 16, 512, 1024), (45, 3, 24, 515, 1056)):
        bank, _, _ = _bank(g, P, n, k)
        x = torch.from_numpy(W.normal_bf16(g, (T, k)).view(np.int16)).cuda().view(torch.bfloat16)
        idx = torch.from_numpy(_idx(g, T, K, P)).cuda()
        want = _product(bank, x, idx, out_dtype=torch.float32)
        out = torch.empty_like(want)
        ws = torch.empty(m.moe_mx_product_workspace_bytes(P, n, k, T, K), dtype=torch.uint8, device="cuda")
        jobs.append((bank, x, idx, want, out, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for bank, x, idx, _, out, ws, s in jobs:
            m.moe_mx_product(bank, x, idx, out, ws, stream=s)
    torch.cuda.synchronize()
    for _, _, _, want, out, _, _ in jobs:
        assert torch.equal(want, out)


@pytest.mark.parametrize("fmt", ["mxfp4", "e2m1"])
def test_rows_past_32_bit_offsets(fmt):
    _say("large rows", fmt)
    rows, cols, B, tail = 2**20 + 77, 4128, 32 if fmt == "mxfp4" else 16, 80   # 4.3e9 elements
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda")
    scales = torch.randint(100, 120, (rows, cols // B), dtype=torch.uint8, device="cuda")
    dst = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    m.moe_dequantize_rows(FMT[fmt], codes, scales, dst)
    few = torch.empty((tail, cols), dtype=torch.bfloat16, device="cuda")
    m.moe_dequantize_rows(FMT[fmt], codes[-tail:].contiguous(), scales[-tail:].contiguous(), few)
    assert torch.equal(dst[-tail:].view(torch.int16), few.view(torch.int16))
    few_codes, few_scales = torch.empty_like(codes[-tail:]), torch.empty_like(scales[-tail:])
    m.moe_quantize_rows(FMT[fmt], few, few_codes, few_scales)
    m.moe_quantize_rows(FMT[fmt], dst, codes, scales)
    torch.cuda.synchronize()
    assert torch.equal(codes[-tail:], few_codes) and torch.equal(scales[-tail:], few_scales)


def test_product_past_32_bit_offsets():
    # one scale to a row and x of E2M1 values in blocks of scale 1: terms are multiples of 1/4 of at
    # most 36, so that their sums are exact in any order, in a bank of few matrices too
    _say("large bank")
    P, n, k, few = 1100, 2048, 4096, 24                                        # 4.6 GB of codes
    assert k * 36 * 4 < 2 ** 24
    codes = torch.randint(0, 256, (P, n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.randint(100, 140, (P, n, 1), dtype=torch.uint8, device="cuda").expand(P, n, k // 32).contiguous()
    g = W.rng(46, "large bank")
    for T, K in ((1, 3), (12, 2), (64, 6)):
        x = ref.VALUES[g.integers(0, 8, (T, k))] * g.choice([-1.0, 1.0], (T, k))
        x[:, ::32] = 6.0
        xt = torch.from_numpy(x).to(torch.bfloat16).cuda()
        idx = torch.from_numpy(g.integers(0, few, (T, K)).astype(np.int32)).cuda()
        got = _product(m.make_mx_bank(codes, scales), xt, idx + (P - few), out_dtype=torch.float32)
        want = _product(m.make_mx_bank(codes[-few:], scales[-few:]), xt, idx, out_dtype=torch.float32)
        assert torch.equal(got, want) and bool(got.any())


def test_operators_run_on_the_given_stream():
    g = W.rng(47, "stream")
    T, P, n, k = 64, 4, 64, 256
    bank, codes, scales = _bank(g, P, n, k)
    idx = torch.from_numpy(_idx(g, T, 1, P, 0.0)).cuda()
    src = torch.from_numpy(W.normal_bf16(g, (T, k)).view(np.int16)).cuda().view(torch.bfloat16)
    want = _product(bank, src, idx, out_dtype=torch.float32)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = torch.zeros_like(src)
    out = torch.empty((T, n), device="cuda")
    ws = torch.empty(m.moe_mx_product_workspace_bytes(P, n, k, T, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        x.copy_(src)
    m.moe_mx_product(bank, x, idx, out, ws, stream=s)   # after the copy, on its stream
    s.synchronize()
    assert torch.equal(out, want)


def test_binding_refuses_what_does_not_fit():
    dev = dict(device="cuda")
    x = torch.zeros((2, 64), dtype=torch.bfloat16, **dev)
    codes, scales = torch.zeros((2, 32), dtype=torch.uint8, **dev), torch.zeros((2, 2), dtype=torch.uint8, **dev)
    ids, w = torch.zeros((2, 4), dtype=torch.int32, **dev), torch.zeros((2, 4), **dev)
    r = m.make_router()
    with pytest.raises(ValueError):
        m.moe_route(r, torch.zeros((2, 8)), 4, ids, w)                      # logits on the host
    with pytest.raises(ValueError):
        m.moe_route(r, torch.zeros((2, 8), dtype=torch.float16, **dev), 4, ids, w)
    with pytest.raises(ValueError):
        m.moe_route(r, torch.zeros((8, 2), **dev).t(), 4, ids, w)           # columns contiguous, not rows
    with pytest.raises(ValueError):
        m.moe_route(r, torch.zeros((2, 8), **dev), 3, ids, w)
    with pytest.raises(ValueError):
        m.moe_route(r, torch.zeros((2, 8), **dev), 4, ids.long(), w)
    with pytest.raises(ValueError):
        m.moe_route(m.make_router(bias=torch.zeros(7, **dev)), torch.zeros((2, 8), **dev), 4, ids, w)
    with pytest.raises(m.MoeError):
        m.moe_route(r, torch.zeros((1, 8), **dev).expand(2, 8), 4, ids, w)  # rows on top of each other
    with pytest.raises(ValueError):
        m.moe_quantize_rows(m.MOE_FMT_MXFP4, x, codes, scales[:, :1])
    with pytest.raises(ValueError):
        m.moe_quantize_rows(m.MOE_FMT_MXFP4, x.half(), codes, scales)
    with pytest.raises(ValueError):
        m.moe_quantize_rows(m.MOE_FMT_E2M1, x, codes, torch.zeros((2, 4), dtype=torch.uint8, **dev),
                            globals=torch.ones(1, **dev), rows_per_global=1)
    with pytest.raises(m.MoeError):
        m.moe_quantize_rows(m.MOE_FMT_MXFP4, x[:, :48], codes, scales)
    bank = m.make_mx_bank(codes.view(1, 2, 32), scales.view(1, 2, 2))
    ws = torch.zeros(1 << 16, dtype=torch.uint8, **dev)
    out = torch.zeros((2, 2), **dev)
    with pytest.raises(ValueError):
        m.moe_mx_product(bank, x[:, :32], None, out, ws)
    with pytest.raises(ValueError):
        m.moe_mx_product(bank, x.float(), None, out, ws)
    with pytest.raises(ValueError):
        m.moe_mx_product(bank, x, ids, out, ws)                             # 8 routes, 2 rows of out
    with pytest.raises(m.MoeError):
        m.moe_mx_product(bank, x, None, out, ws[:256])
    with pytest.raises(ValueError):
        m.make_mx_bank(codes.view(1, 2, 32), scales.view(1, 4, 1))


# ---------------------------------------------------------------- together

def _mx_pool(g, P, H, F):
    banks = [torch.from_numpy(b).cuda() for b in W.mxfp4_expert_rows(g, P, H, F)]
    return m.make_pool(m.MOE_FMT_MXFP4, H, F, P, banks), banks


def _combine(y, idx, w, addend, P):
    """fp32 fma chain over k: the GPU's order, with one rounding a step (in 64 bits: exact products)."""
    T, K = idx.shape
    acc = np.zeros((T, y.shape[1]), np.float32)
    y = y.reshape(T, K, -1)
    for j in range(K):
        live = (idx[:, j] >= 0) & (idx[:, j] < P)
        step = (y[:, j].astype(np.float64) * w[:, j:j + 1].astype(np.float64) + acc).astype(np.float32)
        acc = np.where(live[:, None], step, acc)
    return acc if addend is None else acc + addend


@pytest.mark.parametrize("T,K,P,H,F", [(1, 8, 16, 2048, 512), (1, 2, 4, 64, 128), (5, 3, 4, 96, 32), (40, 2, 6, 320, 160),
                                        (600, 2, 20, 256, 96), (300, 2, 2, 512, 256)])
@pytest.mark.parametrize("with_addend", [False, True])
def test_routed_mx_is_route_product_product_combine(T, K, P, H, F, with_addend):
    _say("routed mx", T, K, P, H, F, with_addend)
    g = W.rng(53, "routed", T, K, P, H, F)
    pool, banks = _mx_pool(g, P, H, F)
    x = torch.from_numpy(W.normal_bf16(g, (T, H)).view(np.int16)).cuda().view(torch.bfloat16)
    logits = torch.from_numpy(g.standard_normal((T, P)).astype(np.float32)).cuda()
    if T > 2:
        logits[1] = -float("inf")
        logits[2, 1:] = float("nan")
    ids = torch.empty((T, K), dtype=torch.int32, device="cuda")
    w = torch.empty((T, K), device="cuda")
    m.moe_route(m.make_router(score=m.MOE_SCORE_SIGMOID, scale=1.5), logits, K, ids, w)
    add = torch.from_numpy((g.standard_normal((T, H)) * 0.01).astype(np.float32)).cuda() if with_addend else None
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((m.moe_routed_mx_workspace_bytes(P, H, F, T, K),), 0xFF, dtype=torch.uint8, device="cuda")
    m.moe_routed_decode_mx(pool, x, ids, w, out, ws, addend=add)
    # the same from the parts, to the bit but for the combine's own rounding
    up = m.make_mx_bank(banks[0].view(P, 2 * F, H // 2), banks[1].view(P, 2 * F, H // 32))
    dn = m.make_mx_bank(banks[2].view(P, H, F // 2), banks[3].view(P, H, F // 32))
    h = _product(up, x, ids, swiglu=True)
    y = _product(dn, h, ids.view(-1, 1), out_dtype=torch.float32)
    torch.cuda.synchronize()
    want = _combine(y.cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), None if add is None else add.cpu().numpy(), P)
    got = _f64(out)
    # fp32 chain against one double-rounded step each: K steps of 2^-24 of the largest partial sum
    slack = (K + 1) * 2.0 ** -23 * (np.abs(w.cpu().numpy()[:, :, None] * y.cpu().numpy().reshape(T, K, H)).sum(1)
                                    + (0 if add is None else np.abs(add.cpu().numpy())))
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + slack).all()
    if T > 2 and add is None:
        assert (out[1] == 0).all()


@pytest.mark.parametrize("T,K,P,H,F", [(4, 6, 30, 2048, 2048), (300, 8, 300, 640, 512), (800, 2, 4, 2048, 11008)])
def test_routed_mx_with_runs_of_two_lengths(T, K, P, H, F):
    # the down product's half as large matrices are taken in runs of another length than the
    # gate/up product's: the lists are made anew, and the result is that of the two alone
    _say("routed mx, two lengths", T, K, P, H, F)
    g = W.rng(54, "two lengths", T, K, P, H, F)
    banks = [torch.from_numpy(g.integers(*r, s, dtype=np.uint8)).cuda().view(-1) for r, s in (
        ((0, 256), (P, 2 * F, H // 2)), ((110, 122), (P, 2 * F, H // 32)), ((0, 256), (P, H, F // 2)),
        ((110, 122), (P, H, F // 32)))]
    pool = m.make_pool(m.MOE_FMT_MXFP4, H, F, P, banks)
    x = torch.from_numpy(W.normal_bf16(g, (T, H)).view(np.int16)).cuda().view(torch.bfloat16)
    ids = torch.from_numpy(_idx(g, T, K, P, 0.02)).cuda()
    w = torch.from_numpy(g.random((T, K), dtype=np.float32)).cuda()
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((m.moe_routed_mx_workspace_bytes(P, H, F, T, K),), 0xFF, dtype=torch.uint8, device="cuda")
    m.moe_routed_decode_mx(pool, x, ids, w, out, ws)
    up = m.make_mx_bank(banks[0].view(P, 2 * F, H // 2), banks[1].view(P, 2 * F, H // 32))
    dn = m.make_mx_bank(banks[2].view(P, H, F // 2), banks[3].view(P, H, F // 32))
    h = _product(up, x, ids, swiglu=True)
    y = _product(dn, h, ids.view(-1, 1), out_dtype=torch.float32)
    torch.cuda.synchronize()
    want = _combine(y.cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), None, P)
    # fp32 chain against one double-rounded step each: K steps of 2^-24 of the largest partial sum
    slack = (K + 1) * 2.0 ** -23 * np.abs(w.cpu().numpy()[:, :, None] * y.cpu().numpy().reshape(T, K, H)).sum(1)
    assert (np.abs(_f64(out) - want) <= 2.0 ** -8 * np.abs(want) + slack).all()


def test_routed_mx_is_near_the_16_bit_activations():
    # quantizing x and h to 4 bits moves the layer's output by about their relative step: E2M1's
    # rounding is uniform within steps of up to 1/4..1/2 of a value, an rms of 0.1 to 0.15 for
    # each of the two, so 0.3 bounds the whole relative 2-norm with room
    g = W.rng(59, "near16")
    T, K, P, H, F = 32, 4, 8, 1024, 256
    pool, _ = _mx_pool(g, P, H, F)
    x = torch.from_numpy(W.normal_bf16(g, (T, H)).view(np.int16)).cuda().view(torch.bfloat16)
    idx = torch.from_numpy(_idx(g, T, K, P, 0.0)).cuda()
    w = torch.full((T, K), 0.25, device="cuda")
    a, b = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(m.moe_routed_mx_workspace_bytes(P, H, F, T, K), dtype=torch.uint8, device="cuda")
    m.moe_routed_decode_mx(pool, x, idx, w, a, ws)
    ws = torch.empty(m.moe_routed_workspace_bytes(2, H, F, T, K), dtype=torch.uint8, device="cuda")
    m.moe_routed_decode(pool, x, idx, w, b, ws)
    torch.cuda.synchronize()
    rel = float((a.double() - b.double()).norm() / b.double().norm())
    assert 0.0 < rel < 0.3, rel


@pytest.mark.parametrize("overlap", [0, 1, 2, 3])
@pytest.mark.parametrize("T", [1, 3, 40])
def test_layer_step_with_a_router(overlap, T):
    import oracle
    from expert_slot_cache_moe_amd.layer import SlotCacheLayers, quantized_banks
    from parity import check_close

    _say("router layer", overlap, T)
    E, S, H, F, K = 16, 12, 64, 128, 3
    g = W.rng(61, "layer", T)
    bf16 = W.bf16_expert_rows(g, E, H, F)
    sh = [(W.normal_bf16(g, 2 * F * H, 0.02), W.normal_bf16(g, H * F, 0.02), W.normal_bf16(g, H, 0.02))]
    bias = torch.from_numpy((g.standard_normal(E) * 0.1).astype(np.float32)).cuda()
    router = m.make_router(score=m.MOE_SCORE_SIGMOID, num_groups=4, top_groups=2, scale=2.0, bias=bias,
                           group_score=m.MOE_GROUP_TOP2)
    lay = SlotCacheLayers(layers=1, experts=E, slots=S, hidden=H, ffn=F, fmt=m.MOE_FMT_MXFP4, host_rows=[bf16],
                          shared=sh, max_tokens=T, max_top_k=K, overlap=overlap, router=router, quantize=True)
    banks = [b.cpu().numpy() for b in quantized_banks(m.MOE_FMT_MXFP4, *bf16, H, F)]
    oc = oracle.OracleCache(1, E, S)
    try:
        for step in range(4):
            x = W.normal_bf16(g, (T, H))
            lg = g.standard_normal((T, E)).astype(np.float32)
            if step == 2:
                lg[0] = -np.inf
            out = torch.empty((T, H), dtype=torch.int16, device="cuda")
            slots = torch.empty((T, K), dtype=torch.int32, device="cuda")
            w = torch.empty((T, K), device="cuda")
            lay.decode(0, torch.from_numpy(x.view(np.int16)).cuda(), torch.from_numpy(lg).cuda(), K, out,
                       ids_out=slots, w_out=w)
            torch.cuda.synchronize()
            ids, e_w = ref.route(lg, K, score="sigmoid", groups=4, top_groups=2, top2=True, scale=2.0, bias=_f64(bias))
            e_slots = oc.admit(0, ids.reshape(-1)).reshape(T, K)
            assert (slots.cpu().numpy() == e_slots).all()
            assert np.allclose(_f64(w), e_w, rtol=1e-6, atol=0)
            _, add = oracle.shared(H, F, *sh[0], x)
            want = oracle.routed(oracle.Pool(2, H, F, banks), np.where(e_slots >= 0, ids, -1), e_w, x, addend=add)
            check_close(out.view(torch.bfloat16).double().cpu().numpy(), want, f"step {step}")
        st = m.moe_cache_read_state(lay.cache)
        assert (st["res"] == oc.res).all() and (st["stats"] == oc.stats).all()
    finally:
        lay.close()


def test_layer_step_without_a_router_is_the_plain_layer_step():
    from expert_slot_cache_moe_amd.layer import SlotCacheLayers

    E, S, H, F, K, T = 8, 8, 64, 128, 2, 1
    g = W.rng(67, "plain layer")
    rows = [W.bf16_expert_rows(g, E, H, F)]
    outs = []
    x = torch.from_numpy(W.normal_bf16(g, (T, H)).view(np.int16)).cuda()
    lg = torch.from_numpy(g.standard_normal((T, E)).astype(np.float32)).cuda()
    for through_router in (False, True):
        lay = SlotCacheLayers(layers=1, experts=E, slots=S, hidden=H, ffn=F, host_rows=rows, max_tokens=T, max_top_k=K)
        out = torch.empty((T, H), dtype=torch.int16, device="cuda")
        if through_router:
            m.moe_layer_decode_router(lay.cache, 0, x, lg, K, out)
        else:
            lay.decode(0, x, lg, K, out)
        torch.cuda.synchronize()
        outs.append(out.clone())
        lay.close()
    assert torch.equal(*outs)


@pytest.mark.parametrize("fmt", ["mxfp4", "e2m1"])
def test_quantized_banks_are_the_plain_rows(fmt):
    from expert_slot_cache_moe_amd.layer import quantized_banks

    E, H, F = 3, 64, 96
    g = W.rng(71, "banks")
    w13, w2 = W.bf16_expert_rows(g, E, H, F)
    w2[1] = 0
    banks = [b.cpu().numpy() for b in quantized_banks(FMT[fmt], w13, w2, H, F)]
    assert [b.shape[1] for b in banks] == m.moe_bank_row_bytes(FMT[fmt], H, F)
    per = 3 if fmt == "e2m1" else 2
    for i, (raw, n, k) in enumerate(((w13, 2 * F, H), (w2, H, F))):
        x = ref.bf16_f64(raw.view(np.uint16)).reshape(E * n, k)
        glob = None
        if fmt == "e2m1":
            glob = banks[per * i + 2].reshape(-1).view(np.float32)
            amax = np.abs(x).reshape(E, -1).max(1)
            assert np.allclose(glob, np.where(amax > 0, amax / 2688, 1.0), rtol=1e-6)
        codes, scales, _ = ref.quantize(x, fmt, glob, n)
        assert (banks[per * i].reshape(E * n, -1) == codes).all()
        assert (banks[per * i + 1].reshape(E * n, -1) == scales).all()
