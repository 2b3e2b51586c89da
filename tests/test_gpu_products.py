"""The route lists, the grouped and dense products and the routed experts of
a prompt on the GPU, against plain 64-bit forms (product_ref.py, where the
bounds are derived).  Inputs that are small whole numbers have sums that fp32
holds exactly in any order: those results are compared for equality."""
import numpy as np
import pytest
import torch

import expert_slot_cache_moe_amd as m
import product_ref as ref
from expert_slot_cache_moe_amd import workloads as W
from expert_slot_cache_moe_amd.layer import SlotCacheLayers

pytestmark = pytest.mark.gpu

ACT = {"none": m.MOE_ACT_NONE, "silu": m.MOE_ACT_SILU, "gelu": m.MOE_ACT_GELU, "swiglu": m.MOE_ACT_SWIGLU}
FORMATS = {"bf16": m.MOE_FMT_BF16, "e2m1": m.MOE_FMT_E2M1, "mxfp4": m.MOE_FMT_MXFP4}
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _say(*a):
    print(*a, flush=True)


def _f64(t):
    return t.double().cpu().numpy()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _name(dtype):
    return str(dtype).split(".")[1]


# ---------------------------------------------------------------- lists

def _lists(idx, P, stream=None):
    T, K = idx.shape
    offsets = torch.full((P + 1,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((T * K,), -7, dtype=torch.int32, device="cuda")
    n = m.moe_group_routes_workspace_bytes(P, T, K)
    ws = torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") if n else None
    m.moe_group_routes(idx, P, offsets, order, ws, stream=stream)
    return offsets, order


@pytest.mark.parametrize("T,K,P", [
    (0, 4, 5), (1, 1, 1), (1, 8, 256), (3, 5, 2), (64, 1, 7), (65, 1, 64), (600, 2, 160), (1024, 1, 1), (1025, 3, 33),
    (2048, 4, 300), (8191, 1, 40), (8193, 1, 40), (4096, 6, 256), (9001, 3, 1), (2777, 7, 4097), (1000, 9, 32768),
    (16384, 10, 512), (100, 64, 2048), (300, 64, 2049), (70000, 9, 130),
])
def test_lists_match_the_plain_form(T, K, P):
    _say("lists", T, K, P)
    g = W.rng(81, "lists", T, K, P)
    idx = np.minimum((g.random((T, K)) ** 2 * P).astype(np.int64), P - 1)
    idx[g.random((T, K)) < 0.05] = -1
    idx[g.random((T, K)) < 0.02] = P
    idx[g.random((T, K)) < 0.01] = -2 ** 31
    idx[g.random((T, K)) < 0.01] = 2 ** 31 - 1
    offsets, order = _lists(_i32(idx), P)
    e_offsets, e_order = ref.lists(idx, P)
    assert (offsets.cpu().numpy() == e_offsets).all()
    assert (order.cpu().numpy() == e_order).all()


@pytest.mark.parametrize("R", [5, 3000, 20000])
@pytest.mark.parametrize("kind", ["one row", "no row", "descending"])
def test_lists_of_uneven_rows(R, kind):
    _say("lists", R, kind)
    P = 97
    idx = {"one row": np.full(R, 41), "no row": np.full(R, -1), "descending": P - 1 - np.arange(R) * P // R}[kind]
    offsets, order = _lists(_i32(idx.reshape(R, 1)), P)
    e_offsets, e_order = ref.lists(idx, P)
    assert (offsets.cpu().numpy() == e_offsets).all() and (order.cpu().numpy() == e_order).all()


# ---------------------------------------------------------------- inputs of the products

def _whole(g, shape, most):
    return torch.from_numpy(g.integers(-most, most + 1, shape).astype(np.float32)).to(torch.bfloat16)


def _bank(g, fmt, P, n, k, whole=False):
    """(bank, weights float64 [P, n, k])."""
    if fmt == "bf16":
        w = (_whole(g, (P, n, k), 2) if whole else
             torch.from_numpy((g.standard_normal((P, n, k)) * 0.05).astype(np.float32)).to(torch.bfloat16)).cuda()
        return m.make_bank(m.MOE_FMT_BF16, w), _f64(w)
    blk = 16 if fmt == "e2m1" else 32
    codes = g.integers(0, 256, (P, n, k // 2)).astype(np.uint8)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(P, n, k)
    v = VALUES[c & 7] * np.where(c & 8, -1.0, 1.0)
    glob = None
    if fmt == "e2m1":
        # E4M3 1, 2 (0x38, 0x40); or anything but NaN
        sc = g.choice([0x38, 0x40], (P, n, k // blk)).astype(np.uint8) if whole else \
            g.integers(0, 0x7f, (P, n, k // blk)).astype(np.uint8)
        e, mant = sc >> 3, sc & 7
        s = np.where(e > 0, (1 + mant / 8) * 2.0 ** (e.astype(float) - 7), mant * 2.0 ** -9)
        glob = np.full(P, 2.0, np.float32) if whole else (0.001 + 0.01 * g.random(P)).astype(np.float32)
        unit = s * glob.astype(np.float64)[:, None, None]
    else:
        sc = g.integers(128, 130, (P, n, k // blk)).astype(np.uint8) if whole else \
            g.integers(115, 130, (P, n, k // blk)).astype(np.uint8)
        unit = 2.0 ** (sc.astype(float) - 127)
    t = lambda a: None if a is None else torch.from_numpy(a).cuda()   # noqa: E731
    return m.make_bank(FORMATS[fmt], t(codes), t(sc), t(glob)), v * np.repeat(unit, blk, axis=2)


def _rows(g, rows, k, whole=False, pad=0):
    x = _whole(g, (rows, k + pad), 2) if whole else \
        torch.from_numpy(g.standard_normal((rows, k + pad)).astype(np.float32)).to(torch.bfloat16)
    return x.cuda()[:, pad // 2:pad // 2 + k]


def _cut(g, R, G):
    """Offsets of G ragged groups over R places, many of them empty, some places in none."""
    cuts = np.sort(g.integers(0, R + 1, G + 1))
    if G > 3:
        cuts[G // 2] = cuts[G // 2 - 1]
    return cuts.astype(np.int32)


def _compare(out, done, val, bnd, whole, fill):
    got = _f64(out)
    assert (got[~done] == fill).all(), "a row that no place names was written"
    if whole:
        assert (got[done] == val[done]).all()
    else:
        assert ref.off(got[done], val[done], bnd[done], _name(out.dtype)) <= 0


GROUPED = [
    # fmt, P, n, k, R, way, act, bias, out
    ("bf16", 3, 1, 1, 5, "rows", "none", True, torch.float32),
    ("bf16", 4, 17, 7, 40, "gather", "silu", False, torch.bfloat16),
    ("bf16", 8, 64, 128, 8, "gather", "swiglu", False, torch.bfloat16),
    ("bf16", 5, 130, 257, 61, "scatter", "gelu", True, torch.float32),
    ("bf16", 24, 515, 1061, 135, "rows", "none", True, torch.float32),
    ("bf16", 6, 96, 130, 700, "gather", "swiglu", True, torch.bfloat16),
    ("bf16", 2, 384, 200, 900, "scatter", "none", False, torch.float32),
    ("bf16", 1, 300, 192, 1000, "rows", "swiglu", False, torch.float32),
    ("bf16", 300, 32, 64, 500, "gather", "none", False, torch.float32),
    ("bf16", 700, 24, 40, 900, "rows", "silu", False, torch.bfloat16),
    ("e2m1", 4, 33, 32, 20, "rows", "none", True, torch.float32),
    ("e2m1", 7, 64, 96, 150, "gather", "swiglu", False, torch.bfloat16),
    ("e2m1", 3, 257, 416, 800, "scatter", "silu", False, torch.float32),
    ("mxfp4", 4, 33, 32, 20, "rows", "none", True, torch.float32),
    ("mxfp4", 7, 64, 96, 150, "gather", "swiglu", False, torch.bfloat16),
    ("mxfp4", 3, 257, 416, 800, "scatter", "gelu", True, torch.float32),
]


def _grouped_case(g, fmt, P, n, k, R, way, act, bias, out_dtype, whole, pad=0):
    bank, w = _bank(g, fmt, P, n, k, whole)
    K = 3 if way == "gather" and R % 3 == 0 else 1
    x = _rows(g, R // K if way == "gather" else R, k, whole, pad)
    G = P if way != "rows" else P + 2
    offsets = _cut(g, R, G)
    order = g.permutation(R).astype(np.int32)
    kw, rkw = {}, {}
    if way == "gather":
        kw, rkw = dict(gather=_i32(order), gather_div=K), dict(gather=order, div=K)
    if way == "scatter":
        kw, rkw = dict(scatter=_i32(order)), dict(scatter=order)
    if way == "rows":
        mats = g.integers(-1, P + 1, G).astype(np.int32)
        kw, rkw = dict(matrices=_i32(mats)), dict(matrices=mats)
    b = None
    if bias:
        b = g.integers(-4, 5, (P, n)) if whole else g.standard_normal((P, n))
        b = torch.from_numpy(b.astype(np.float32)).to(torch.bfloat16 if n % 2 else torch.float32).cuda()
    cols = n // 2 if act == "swiglu" else n
    out = torch.full((R, cols + pad), 77.0, dtype=out_dtype, device="cuda")
    view = out[:, pad // 2:pad // 2 + cols]
    m.moe_grouped_product(bank, x, _i32(offsets), view, activation=ACT[act], bias=b, **kw)
    done, val, bnd = ref.grouped(w, _f64(x), offsets, R, R=R, act=act, bias=None if b is None else _f64(b), **rkw)
    _compare(view, done, val, bnd, whole and act == "none", 77.0)
    if pad:
        assert (out[:, :pad // 2] == 77.0).all() and (out[:, pad // 2 + cols:] == 77.0).all()


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "-".join(str(v) for v in c))
def test_grouped_product_matches_the_plain_form(case):
    _say("grouped", case)
    _grouped_case(W.rng(82, "grouped", *case[:-1]), *case, whole=False)


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "-".join(str(v) for v in c))
def test_grouped_product_of_whole_numbers_is_exact(case):
    case = case[:6] + ("none", case[7], torch.float32)
    _say("grouped whole", case)
    _grouped_case(W.rng(83, "whole", *case[:-1]), *case, whole=True, pad=6)


def _linear_case(g, fmt, T, n, k, act, bias, residual, out_dtype, whole, pad=0):
    bank, w = _bank(g, fmt, 1, n, k, whole)
    x = _rows(g, T, k, whole, pad)
    cols = n // 2 if act == "swiglu" else n
    b = torch.from_numpy((g.integers(-4, 5, n) if whole else g.standard_normal(n)).astype(np.float32)).cuda() if bias else None
    res = None
    if residual is not None:
        res = _rows(g, T, cols, whole, pad).to(residual)
    out = torch.full((T, cols + pad), 77.0, dtype=out_dtype, device="cuda")
    view = out[:, :cols]
    m.moe_linear(bank, x, view, activation=ACT[act], bias=b, residual=res)
    val, bnd = ref.product(w[0], _f64(x), act, None if b is None else _f64(b), None if res is None else _f64(res))
    _compare(view, np.ones(T, bool), val, bnd, whole and act == "none", 77.0)
    if pad:
        assert (out[:, cols:] == 77.0).all()


LINEAR = [
    # fmt, T, n, k, act, bias, residual, out
    ("bf16", 1, 1, 1, "none", True, torch.float32, torch.float32),
    ("bf16", 1, 256, 2048, "none", True, None, torch.float32),
    ("bf16", 2, 66, 300, "swiglu", True, torch.bfloat16, torch.bfloat16),
    ("bf16", 15, 40, 129, "silu", False, torch.float32, torch.bfloat16),
    ("bf16", 17, 515, 1061, "gelu", True, torch.bfloat16, torch.bfloat16),
    ("bf16", 77, 200, 136, "none", False, torch.bfloat16, torch.float32),
    ("bf16", 129, 260, 72, "swiglu", False, None, torch.float32),
    ("bf16", 300, 512, 1024, "gelu", True, torch.bfloat16, torch.bfloat16),
    ("bf16", 600, 1024, 256, "none", False, torch.bfloat16, torch.bfloat16),
    ("bf16", 1000, 130, 65, "silu", True, torch.float32, torch.float32),
    ("bf16", 1500, 600, 190, "swiglu", True, torch.bfloat16, torch.bfloat16),
    ("e2m1", 1, 64, 256, "none", False, None, torch.float32),
    ("e2m1", 200, 520, 352, "silu", True, torch.bfloat16, torch.bfloat16),
    ("mxfp4", 3, 130, 160, "swiglu", False, None, torch.bfloat16),
    ("mxfp4", 1100, 264, 288, "none", True, torch.float32, torch.float32),
]


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(str(v) for v in c))
def test_linear_matches_the_plain_form(case):
    _say("linear", case)
    _linear_case(W.rng(84, "linear", *case[:6]), *case, whole=False)


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(str(v) for v in c))
def test_linear_of_whole_numbers_is_exact(case):
    case = case[:4] + ("none",) + case[5:7] + (torch.float32,)
    _say("linear whole", case)
    _linear_case(W.rng(85, "whole", *case[:6]), *case, whole=True, pad=6)


def test_residual_may_be_the_output():
    g = W.rng(86, "inplace")
    for T, n, k in ((3, 64, 64), (700, 320, 96)):
        bank, w = _bank(g, "bf16", 1, n, k)
        x, y = _rows(g, T, k), _rows(g, T, n).contiguous()
        before = _f64(y)
        m.moe_linear(bank, x, y, residual=y)
        val, bnd = ref.product(w[0], _f64(x), residual=before)
        assert ref.off(_f64(y), val, bnd, "bfloat16") <= 0


# ---------------------------------------------------------------- what must not leak

@pytest.mark.parametrize("T", [1, 40, 300])
def test_nan_and_infinity_stay_in_their_rows(T):
    """A row of x, or of a matrix, with NaN or infinity reaches its own outputs only, at widths whose last
    step of k is cut off in the middle."""
    g = W.rng(87, "nan", T)
    P, n, k = 3, 70, 203
    w = torch.from_numpy(g.standard_normal((P, n, k)).astype(np.float32)).to(torch.bfloat16).cuda()
    w[0, 5, 202] = float("nan")
    w[1, 0, 0] = float("inf")                 # right behind the end of matrix 0
    x = _rows(g, 3 * T, k).contiguous()
    x[0, 0] = float("nan")
    x[3 * T - 1, 202] = -float("inf")
    offsets = _i32([0, T, 2 * T, 3 * T])
    out = torch.zeros((3 * T, n), dtype=torch.float32, device="cuda")
    m.moe_grouped_product(m.make_bank(m.MOE_FMT_BF16, w), x, offsets, out)
    e = np.zeros((3 * T, n))
    for i in range(3):
        with np.errstate(invalid="ignore"):
            e[i * T:(i + 1) * T] = _f64(x[i * T:(i + 1) * T]) @ _f64(w[i]).T
    got = _f64(out)
    assert (np.isnan(got) == np.isnan(e)).all()
    assert (np.isinf(got) == np.isinf(e)).all()
    inf = np.isinf(e)
    assert (got[inf] == e[inf]).all()


@pytest.mark.parametrize("fmt,bad", [("e2m1", 0x7f), ("mxfp4", 0xff)])
@pytest.mark.parametrize("R", [2, 600])
def test_nan_scales_reach_their_outputs_alone(fmt, bad, R):
    g = W.rng(88, "nan scale", fmt, R)
    n, k = 48, 96
    bank, w = _bank(g, fmt, 2, n, k)
    bank._keep[1][1, 7, 1] = bad
    x = _rows(g, R, k)
    out = torch.zeros((R, n), dtype=torch.float32, device="cuda")
    m.moe_grouped_product(bank, x, _i32([0, R // 2, R]), out)
    got = _f64(out)
    nan = np.zeros((R, n), bool)
    nan[R // 2:, 7] = True
    assert (np.isnan(got) == nan).all()


def test_indices_out_of_range_are_left_out():
    g = W.rng(89, "range")
    for R in (30, 900):
        bank, w = _bank(g, "bf16", 4, 40, 64)
        x = _rows(g, 20, 64)
        offsets = np.array([-5, R // 4, R // 2, R // 2, R + 9], np.int32)
        gather = g.integers(-30, 90, R).astype(np.int32)
        scatter = (g.permutation(R) - 5).astype(np.int32)
        out = torch.full((R - 10, 40), 77.0, dtype=torch.float32, device="cuda")
        m.moe_grouped_product(bank, x, _i32(offsets), out, gather=_i32(gather), gather_div=3, scatter=_i32(scatter))
        done, val, bnd = ref.grouped(w, _f64(x), offsets, R - 10, gather=gather, div=3, scatter=scatter, R=R)
        _compare(out, done, val, bnd, False, 77.0)


def test_offsets_that_do_not_ascend_stay_in_bounds():
    g = W.rng(90, "descending")
    bank, _ = _bank(g, "bf16", 4, 40, 64)
    x = _rows(g, 50, 64)
    out = torch.full((50, 40), 77.0, dtype=torch.float32, device="cuda")
    m.moe_grouped_product(bank, x, _i32([40, 10, 2 ** 31 - 1, -2 ** 31, 20]), out)
    torch.cuda.synchronize()
    assert (out[:10] == 77.0).all() or torch.isfinite(out).all()


def test_a_places_result_depends_on_its_matrix_and_x_alone():
    """One row of x in many places of groups that share a matrix: equal bits."""
    g = W.rng(91, "places")
    for R, n, k in ((60, 48, 200), (2000, 300, 200)):
        w1 = torch.from_numpy(g.standard_normal((1, n, k)).astype(np.float32)).to(torch.bfloat16)
        bank = m.make_bank(m.MOE_FMT_BF16, w1.repeat(5, 1, 1).contiguous().cuda())
        x = _rows(g, 1, k)
        out = torch.zeros((R, n), dtype=torch.float32, device="cuda")
        m.moe_grouped_product(bank, x, _i32([0, 1, R // 3, R // 3 + 17, R - 1, R]), out,
                              gather=_i32(np.zeros(R)))
        assert (out == out[0]).all()


# ---------------------------------------------------------------- streams, graphs, large buffers

def test_captured_products_replay():
    g = W.rng(92, "graph")
    T, K, P, H, F = 40, 3, 12, 128, 96
    banks = [_bank(g, "bf16", P, 2 * F, H)[0], _bank(g, "mxfp4", P, H, F)[0]]
    dense, _ = _bank(g, "bf16", 1, 64, H)
    x, idx = _rows(g, T, H), _i32(g.integers(-1, P, (T, K)))
    offsets, order = (torch.empty(s, dtype=torch.int32, device="cuda") for s in (P + 1, T * K))
    h = torch.zeros((T * K, F), dtype=torch.bfloat16, device="cuda")
    d = torch.zeros((T * K, H), dtype=torch.float32, device="cuda")
    y = torch.zeros((T, 64), dtype=torch.bfloat16, device="cuda")

    def step():
        m.moe_group_routes(idx, P, offsets, order)
        m.moe_grouped_product(banks[0], x, offsets, h, gather=order, gather_div=K, activation=m.MOE_ACT_SWIGLU)
        m.moe_grouped_product(banks[1], h, offsets, d, scatter=order)
        m.moe_linear(dense, x, y, activation=m.MOE_ACT_GELU)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(_rows(g, T, H))
        idx.copy_(_i32(g.integers(-1, P, (T, K))))
        h.zero_(), d.zero_(), y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (offsets, order, h, d, y)]
        h.zero_(), d.zero_(), y.zero_()
        step()
        for a, b in zip(got, (offsets, order, h, d, y)):
            assert torch.equal(a, b), i


def test_products_on_two_streams_at_once():
    g = W.rng(93, "streams")
    n, k, R, P = 200, 160, 500, 9
    work = []
    for i in range(2):
        bank, w = _bank(g, ("bf16", "e2m1")[i], P, n, k)
        x, offsets = _rows(g, R, k), _cut(g, R, P)
        work.append((bank, w, x, offsets, _i32(offsets), torch.full((R, n), 77.0, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for bank, _, x, _, off, out, s in work:
            m.moe_grouped_product(bank, x, off, out, stream=s)
    torch.cuda.synchronize()
    for _, w, x, offsets, _, out, _ in work:
        done, val, bnd = ref.grouped(w, _f64(x), offsets, R)
        _compare(out, done, val, bnd, False, 77.0)


def test_matrices_and_rows_past_32_bit_offsets():
    """Matrices past 4 GiB into their bank, rows of x and out past 4 GiB into theirs."""
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GiB of device memory")
    g = W.rng(94, "large")
    P, n, k = 700, 2048, 2048                # 5.9 GB
    w = torch.zeros((P, n, k), dtype=torch.bfloat16, device="cuda")
    some = [0, 511, 699]
    for i in some:
        w[i] = torch.from_numpy((g.standard_normal((n, k)) * 0.05).astype(np.float32)).to(torch.bfloat16)
    bank = m.make_bank(m.MOE_FMT_BF16, w)
    stride = 1 << 22
    for R in (6, 700):
        xb = torch.zeros((R, stride), dtype=torch.bfloat16, device="cuda")
        ob = torch.zeros((R, stride), dtype=torch.bfloat16, device="cuda")
        x, out = xb[:, stride - k:], ob[:, stride - n:]
        x.copy_(_rows(g, R, k))
        m.moe_grouped_product(bank, x, _i32([0, R // 3, R // 2, R]), out, matrices=_i32(some))
        done, val, bnd = ref.grouped(np.stack([_f64(w[i]) for i in some]), _f64(x), [0, R // 3, R // 2, R], R)
        _compare(out, done, val, bnd, False, 0.0)
        assert not ob[:, :stride - n].any()


# ---------------------------------------------------------------- the binding

def test_binding_refuses_what_does_not_fit():
    g = W.rng(95, "binding")
    bank, _ = _bank(g, "bf16", 3, 32, 64)
    one, _ = _bank(g, "bf16", 1, 32, 64)
    x, out, off = _rows(g, 8, 64), torch.zeros((8, 32), device="cuda"), _i32([0, 2, 4, 8])
    bad = [
        lambda: m.moe_grouped_product(bank, x.float(), off, out),
        lambda: m.moe_grouped_product(bank, x[:, :32], off, out),
        lambda: m.moe_grouped_product(bank, x.cpu(), off, out),
        lambda: m.moe_grouped_product(bank, x, off.long(), out),
        lambda: m.moe_grouped_product(bank, x, off, out[:, :16]),
        lambda: m.moe_grouped_product(bank, x, off, out.to(torch.float16)),
        lambda: m.moe_grouped_product(bank, x, off, out, matrices=_i32([0, 1])),
        lambda: m.moe_grouped_product(bank, x, off, out, bias=torch.zeros(32, device="cuda")),
        lambda: m.moe_grouped_product(bank, x, off, out, gather=_i32(range(8)), scatter=_i32(range(4))),
        lambda: m.moe_linear(bank, x, out),
        lambda: m.moe_linear(one, x, out[:4]),
        lambda: m.moe_linear(one, x, out, residual=out[:4]),
        lambda: m.moe_linear(one, x, out, bias=torch.zeros((1, 32), device="cuda")),
        lambda: m.moe_linear(one, x.t(), out),
        lambda: m.moe_group_routes(_i32([[0, 1]]), 4, _i32(range(4)), _i32(range(2))),
        lambda: m.moe_group_routes(_i32([0, 1]), 4, _i32(range(5)), _i32(range(2))),
        lambda: m.make_bank(m.MOE_FMT_BF16, torch.zeros((2, 4, 8), device="cuda")),
        lambda: m.make_bank(m.MOE_FMT_MXFP4, torch.zeros((2, 4, 16), dtype=torch.uint8, device="cuda")),
        lambda: m.make_bank(m.MOE_FMT_BF16, torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, m.MoeError)):
            call()
            pytest.fail(f"call {i} was taken")


# ---------------------------------------------------------------- the routed experts of a prompt

def _combine(y, idx, w, addend, P):
    """y fp32 [T, K, H] -> bf16 [T, H], added as the combine documents it."""
    T, K = idx.shape
    out = np.zeros((T, y.shape[2]), np.float64)
    for j in range(K):
        ok = ((idx[:, j] >= 0) & (idx[:, j] < P))[:, None]
        out = out + np.where(ok, w[:, j:j + 1] * y[:, j], 0.0)
    return out + (0 if addend is None else addend)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1", "mxfp4"])
@pytest.mark.parametrize("T,K,P,H,F,with_addend", [
    (1, 8, 32, 128, 64, True), (5, 2, 3, 64, 96, False), (300, 4, 16, 256, 128, True), (1500, 6, 9, 128, 160, False),
])
def test_routed_prefill_is_lists_products_combine(fmt, T, K, P, H, F, with_addend):
    _say("prefill", fmt, T, K, P, H, F)
    g = W.rng(96, "prefill", fmt, T, K, P, H, F)
    (up, w13), (down, w2) = _bank(g, fmt, P, 2 * F, H), _bank(g, fmt, P, H, F)
    banks = [t.view(P, -1).view(torch.uint8) for b in (up, down) for t in b._keep]
    pool = m.make_pool(FORMATS[fmt], H, F, P, banks)
    x = _rows(g, T, H).contiguous()
    idx = g.integers(0, P, (T, K)).astype(np.int32)
    idx[g.random((T, K)) < 0.1] = -1
    idx[g.random((T, K)) < 0.02] = P
    w = torch.from_numpy(g.random((T, K)).astype(np.float32)).cuda()
    add = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).cuda() if with_addend else None
    out = torch.full((T, H), 77.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((m.moe_routed_prefill_workspace_bytes(FORMATS[fmt], P, H, F, T, K),), 0x7f, dtype=torch.uint8,
                    device="cuda")
    m.moe_routed_prefill(pool, x, _i32(idx), w, out, ws, addend=add)
    # the same in its parts
    offsets, order = _lists(_i32(idx), P)
    h = torch.zeros((T * K, F), dtype=torch.bfloat16, device="cuda")
    d = torch.zeros((T * K, H), dtype=torch.float32, device="cuda")
    m.moe_grouped_product(up, x, offsets, h, gather=order, gather_div=K, activation=m.MOE_ACT_SWIGLU)
    m.moe_grouped_product(down, h, offsets, d, scatter=order)
    # each part against its plain form
    e_off, e_order = ref.lists(idx, P)
    done, val, bnd = ref.grouped(w13, _f64(x), e_off, T * K, gather=e_order, div=K, R=T * K, act="swiglu")
    assert ref.off(_f64(h)[done], val[done], bnd[done], "bfloat16") <= 0
    done, val, bnd = ref.grouped(w2, _f64(h), e_off, T * K, scatter=e_order)
    assert ref.off(_f64(d)[done], val[done], bnd[done], "float32") <= 0
    # the combine adds K products and an addend in fp32
    a = None if add is None else _f64(add)
    y = _f64(d).reshape(T, K, H)
    e = _combine(y, idx, _f64(w), a, P)
    mag = _combine(np.abs(y), idx, _f64(w), None if a is None else np.abs(a), P)
    assert (np.abs(_f64(out) - e) <= mag * (2 * K + 2) * 2.0 ** -24 + np.abs(e) * 2.0 ** -8 + 2.0 ** -133).all()


@pytest.mark.parametrize("fmt", [m.MOE_FMT_BF16, m.MOE_FMT_E2M1, m.MOE_FMT_MXFP4])
def test_routed_prefill_is_near_routed_decode(fmt):
    """The same experts and roundings in another order of the sums."""
    T, K, P, H, F = 700, 4, 24, 1024, 256
    g = W.rng(97, "near", fmt)
    banks = W.device_expert_rows(fmt, (97, "near"), P, H, F)
    pool = m.make_pool(fmt, H, F, P, banks)
    x = torch.from_numpy(W.normal_bf16(g, (T, H)).view(np.int16)).cuda().view(torch.bfloat16)
    idx = _i32(np.stack([g.choice(P, K, replace=False) for _ in range(T)]))
    w = torch.from_numpy(g.random((T, K)).astype(np.float32)).cuda()
    outs = []
    for fn, n in ((m.moe_routed_prefill, m.moe_routed_prefill_workspace_bytes(fmt, P, H, F, T, K)),
                  (m.moe_routed_decode, m.moe_routed_workspace_bytes(fmt, H, F, T, K))):
        out = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
        fn(pool, x, idx, w, out, torch.empty(n, dtype=torch.uint8, device="cuda"))
        outs.append(_f64(out))
    # an activation that rounds the other way moves a sum by one of its F terms' 2^-8
    assert np.abs(outs[0] - outs[1]).max() <= 2.0 ** -6 * np.abs(outs[1]).max()


def test_layers_prefill_through_the_streamed_experts():
    """SlotCacheLayers.prefill: every token's experts, whatever the cache holds, and the shared expert."""
    L, E, H, F, T, K = 2, 12, 128, 64, 90, 3
    g = W.rng(98, "layers")
    rows = [W.expert_rows(m.MOE_FMT_BF16, W.rng(98, "rows", l), E, H, F) for l in range(L)]
    shared = [(W.normal_bf16(g, (2 * F * H,), 0.02), W.normal_bf16(g, (H * F,), 0.02), W.normal_bf16(g, (H,), 0.02)),
              None]
    lay = SlotCacheLayers(layers=L, experts=E, slots=4, hidden=H, ffn=F, host_rows=rows, shared=shared, max_tokens=T,
                          max_top_k=K, router=[None, m.make_router(score=m.MOE_SCORE_SIGMOID)])
    try:
        for l in range(L):
            x = torch.from_numpy(W.normal_bf16(g, (T, H)).view(np.int16)).cuda().view(torch.bfloat16)
            logits = torch.from_numpy(g.standard_normal((T, E)).astype(np.float32)).cuda()
            out = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
            ids = torch.zeros((T, K), dtype=torch.int32, device="cuda")
            w = torch.zeros((T, K), dtype=torch.float32, device="cuda")
            lay.prefill(l, x, logits, K, out, ids_out=ids, w_out=w)
            e_ids, e_w = torch.zeros_like(ids), torch.zeros_like(w)
            if l == 0:
                m.moe_topk(logits, K, e_ids, e_w)
            else:
                m.moe_route(lay.routers[1], logits, K, e_ids, e_w)
            assert torch.equal(ids, e_ids) and torch.equal(w, e_w)
            # against moe_routed_decode over the same experts
            add = None
            if shared[l] is not None:
                add = torch.zeros((T, H), dtype=torch.float32, device="cuda")
                m.moe_shared_expert(lay.shared[l], H, x, add, torch.empty(
                    m.moe_routed_workspace_bytes(m.MOE_FMT_BF16, H, F, T, 1), dtype=torch.uint8, device="cuda"))
            e = torch.zeros_like(out)
            m.moe_routed_decode(lay.streamed_pool(l), x, ids, w, e, torch.empty(
                m.moe_routed_workspace_bytes(m.MOE_FMT_BF16, H, F, T, K), dtype=torch.uint8, device="cuda"),
                addend=add)
            assert np.abs(_f64(out) - _f64(e)).max() <= 2.0 ** -6 * np.abs(_f64(e)).max()
    finally:
        lay.close()


@pytest.mark.parametrize("T,K,P", [(1 << 16, 64, 300), (1 << 19, 8, 4095), (1 << 18, 4, 4096)])
def test_lists_of_many_routes(T, K, P):
    """Up to the most routes, on both sides of the rows that waves count alone."""
    _say("many lists", T, K, P)
    g = W.rng(99, "many", T, P)
    idx = (g.random((T, K)) ** 3 * (P + 1)).astype(np.int32) - 1
    offsets, order = _lists(_i32(idx), P)
    key = np.where(idx.reshape(-1) < 0, P, idx.reshape(-1))
    assert (offsets.cpu().numpy() == np.searchsorted(np.sort(key), np.arange(P + 1))).all()
    assert (order.cpu().numpy() == np.argsort(key, kind="stable")).all()
