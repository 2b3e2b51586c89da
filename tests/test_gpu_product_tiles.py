"""The tiles of many places at every kind of stage: one, two and more whole
stages of k, and a last one that is cut off; with everything that an epilogue
does.  Each case names the form that it is to reach (product_forms.py).
Whole numbers, whose sums fp32 holds in any order, are compared for equality;
the bounds of the others: activation_ref.py."""
import numpy as np
import pytest
import torch

import activation_ref as aref
import expert_slot_cache_moe_amd as m
import product_forms as forms
import product_ref as ref
from expert_slot_cache_moe_amd import workloads as W

pytestmark = pytest.mark.gpu

ACT = {"none": m.MOE_ACT_NONE, "silu": m.MOE_ACT_SILU, "gelu": m.MOE_ACT_GELU, "swiglu": m.MOE_ACT_SWIGLU}
F32, BF16 = torch.float32, torch.bfloat16


def _f64(t):
    return t.double().cpu().numpy()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _values(g, shape, whole, scale=1.0):
    v = g.integers(-2, 3, shape) if whole else g.standard_normal(shape, np.float32) * np.float32(scale)
    return torch.from_numpy(v.astype(np.float32)).to(BF16).cuda()


def _off(out, val, bnd, exact):
    got = _f64(out)
    if exact:
        return 0.0 if (got == val).all() else float(np.abs(got - val).max())
    return ref.off(got, val, bnd, str(out.dtype).split(".")[1])


DENSE = {forms.TILE64: (4100, 500), forms.TILE128: (8200, 500), forms.TILE256: (65600, 200)}
# one stage, two, three, more; a cut second, fourth and seventeenth; rows that begin at any element
STAGES = [64, 72, 128, 192, 203, 448, 1061]
EPILOGUES = [
    # act, bias, residual, out, the residual is out
    ("none", True, None, F32, False), ("silu", True, BF16, BF16, False), ("gelu", False, F32, F32, False),
    ("none", False, BF16, BF16, True), ("gelu", True, BF16, F32, False), ("silu", False, F32, F32, True),
    ("swiglu", True, F32, BF16, False), ("swiglu", False, BF16, F32, False),
]


@pytest.mark.parametrize("k", STAGES)
@pytest.mark.parametrize("form", DENSE, ids=lambda f: forms.NAMES[f])
def test_dense_tiles_of_whole_numbers_are_exact(form, k):
    T, n = DENSE[form]
    i = STAGES.index(k)
    pad = (0, 6, 3)[i % 3]
    print("dense whole", T, n, k, pad, flush=True)
    g = W.rng(140, form, k)
    w, x = _values(g, (1, n, k), True), _values(g, (T, k + pad), True)[:, :k]
    assert forms.form_of("bf16", n, k, T, x_stride=k + pad) == form
    bias = torch.from_numpy(g.integers(-9, 10, n).astype(np.float32)).cuda() if i % 2 else None
    residual = (None, BF16, F32)[(i + form) % 3]
    big = torch.full((T + 2, n + pad), 77.0, device="cuda")
    out = big[1:T + 1, :n]
    res = None
    if residual is F32 and i % 2:
        out.copy_(_values(g, (T, n), True))
        res = out
    elif residual is not None:
        res = _values(g, (T, n + pad), True).to(residual)[:, :n]
    before = None if res is None else _f64(res)
    m.moe_linear(m.make_bank(m.MOE_FMT_BF16, w), x, out, bias=bias, residual=res)
    val = _f64(x) @ _f64(w[0]).T + (0 if bias is None else _f64(bias)) + (0 if before is None else before)
    assert _off(out, val, None, True) == 0
    assert (big[0] == 77).all() and (big[T + 1] == 77).all() and (big[:, n:] == 77).all()


@pytest.mark.parametrize("epilogue", range(len(EPILOGUES)))
@pytest.mark.parametrize("form", DENSE, ids=lambda f: forms.NAMES[f])
def test_dense_tiles_with_every_epilogue(form, epilogue):
    act, with_bias, residual, dtype, in_place = EPILOGUES[epilogue]
    k = STAGES[(epilogue + form) % 6 + 1]                # more than one stage
    (T, cols), pad = DENSE[form], (0, 5, 8)[epilogue % 3]
    n = 2 * cols if act == "swiglu" else cols
    if act == "swiglu" and form != forms.TILE256:
        n, cols = cols, cols // 2
    print("dense", act, with_bias, residual, dtype, T, n, k, pad, flush=True)
    assert forms.form_of("bf16", n, k, T, swiglu=act == "swiglu", x_stride=k + pad) == form
    g = W.rng(141, form, epilogue)
    w, x = _values(g, (1, n, k), False, 1 / np.sqrt(k)), _values(g, (T, k + pad), False)[:, :k]
    bias = torch.from_numpy(g.standard_normal(n).astype(np.float32)).cuda() if with_bias else None
    out = torch.full((T, cols + pad), 77.0, dtype=dtype, device="cuda")
    res = None
    if residual is not None:
        res = _values(g, (T, cols + pad), False).to(residual)[:, :cols]
        if in_place:
            out[:, :cols] = res
    before = None if res is None else _f64(res)
    view = out[:, :cols]
    m.moe_linear(m.make_bank(m.MOE_FMT_BF16, w), x, view, activation=ACT[act], bias=bias,
                 residual=view if in_place else res)
    val, bnd = aref.product(_f64(w[0]), _f64(x), act, None if bias is None else _f64(bias), before)
    assert _off(view, val, bnd, False) <= 0
    assert (out[:, cols:] == 77).all()


GROUPED = {forms.TILE64: (8, 500, 2000), forms.TILE128: (8, 1000, 2000), forms.TILE256: (8, 1000, 8000)}


@pytest.mark.parametrize("k", STAGES)
@pytest.mark.parametrize("form", GROUPED, ids=lambda f: forms.NAMES[f])
def test_grouped_tiles_of_whole_numbers_are_exact(form, k):
    """Ragged groups over matrices in another order, some of them not there, gathered rows and scattered results."""
    P, n, R = GROUPED[form]
    i = STAGES.index(k)
    pad = (6, 0, 3)[i % 3]
    print("grouped whole", P, n, k, R, pad, flush=True)
    g = W.rng(142, form, k)
    assert forms.form_of("bf16", n, k, R, groups=P, x_stride=k + pad) == form
    w, x = _values(g, (P, n, k), True), _values(g, (R // 2, k + pad), True)[:, :k]
    cuts = np.sort(g.integers(0, R + 1, P + 1)).astype(np.int32)
    cuts[P // 2] = cuts[P // 2 - 1]
    gather, scatter = g.integers(-3, 2 * (R // 2) + 3, R).astype(np.int32), g.permutation(R).astype(np.int32) - 3
    mats = g.permutation(P).astype(np.int32)
    mats[g.integers(0, P)] = -1
    bias = torch.from_numpy(g.integers(-9, 10, (P, n)).astype(np.float32)).cuda() if i % 2 else None
    big = torch.full((R + 2, n + pad), 77.0, device="cuda")
    out = big[1:R + 1, :n]
    m.moe_grouped_product(m.make_bank(m.MOE_FMT_BF16, w), x, _i32(cuts), out, matrices=_i32(mats), gather=_i32(gather),
                          gather_div=2, scatter=_i32(scatter), bias=bias)
    done, val, _ = ref.grouped(_f64(w), _f64(x), cuts, R, matrices=mats, gather=gather, div=2, scatter=scatter, R=R,
                               bias=None if bias is None else _f64(bias))
    got = _f64(out)
    assert done.any() and (got[done] == val[done]).all() and (got[~done] == 77).all()
    assert (big[0] == 77).all() and (big[R + 1] == 77).all() and (big[:, n:] == 77).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
@pytest.mark.parametrize("form", GROUPED, ids=lambda f: forms.NAMES[f])
def test_grouped_tiles_with_activations(form, act):
    P, n, R = GROUPED[form]
    k = (203, 192, 136)[("silu", "gelu", "swiglu").index(act)]
    cols = n // 2 if act == "swiglu" else n
    assert forms.form_of("bf16", n, k, R, groups=P, swiglu=act == "swiglu") == form
    g = W.rng(143, form, act)
    w, x = _values(g, (P, n, k), False, 1 / np.sqrt(k)), _values(g, (R, k), False)
    bias = torch.from_numpy(g.standard_normal((P, n)).astype(np.float32)).cuda()
    cuts = np.concatenate([[0], np.sort(g.integers(0, R + 1, P - 1)), [R]]).astype(np.int32)
    out = torch.full((R, cols), 77.0, dtype=BF16, device="cuda")
    m.moe_grouped_product(m.make_bank(m.MOE_FMT_BF16, w), x, _i32(cuts), out, activation=ACT[act], bias=bias)
    for p in range(P):
        s = slice(cuts[p], cuts[p + 1])
        val, bnd = aref.product(_f64(w[p]), _f64(x[s]), act, _f64(bias[p]))
        assert _off(out[s], val, bnd, False) <= 0


@pytest.mark.parametrize("form", DENSE, ids=lambda f: forms.NAMES[f])
def test_shared_prefill_whose_gated_products_take_tiles(form):
    """The down product, whose sums are taken times the gate's factor, in the tiles of 64, 128 and 256 places."""
    T, H = DENSE[form]
    F = 203 if form != forms.TILE256 else 136
    print("shared", T, H, F, flush=True)
    assert forms.form_of("bf16", H, F, T) == form
    g = W.rng(144, form)
    w13, w2, gate = (_values(g, s, False, 0.1) for s in ((2 * F, H), (H, F), (H,)))
    x = _values(g, (T, H), False)
    big = torch.full((T + 2, H), 77.0, device="cuda")
    sh = m.make_shared(w13.view(-1).view(torch.int16), w2.view(-1).view(torch.int16), gate.view(torch.int16), ffn=F)
    ws = torch.full((m.moe_shared_prefill_workspace_bytes(H, F, T),), 0x7f, dtype=torch.uint8, device="cuda")
    m.moe_shared_prefill(sh, H, x, big[1:T + 1], ws)
    h, dh = aref.product(_f64(w13), _f64(x), "swiglu")
    dh = dh + (np.abs(h) + dh) * 2.0 ** -8 + 2.0 ** -133                # and its rounding to bf16
    a2 = np.abs(_f64(w2)).T
    y, dy = h @ _f64(w2).T, dh @ a2 + F * 2.0 ** -23 * ((np.abs(h) + dh) @ a2)
    logit, dl = ref.product(_f64(gate)[None], _f64(x))
    s = 1 / (1 + np.exp(-logit))
    # the sigmoid's slope is at most 1/4; the rest as silu's in activation_ref
    ds = dl / 4 + (2.0 ** -21 + np.abs(logit) * 2.0 ** -23) * s + 2.0 ** -126
    bound = (s + ds) * dy + ds * np.abs(y) + 2.0 ** -23 * np.abs(s * y)
    assert (np.abs(_f64(big[1:T + 1]) - s * y) <= bound).all()
    assert (big[0] == 77).all() and (big[T + 1] == 77).all()


# ---------------------------------------------------------------- offsets that do not ascend

# format, columns, k, places over four groups, form
CLIPPED = [("bf16", 40, 64, 50, forms.SPLIT), ("bf16", 400, 200, 1600, forms.TILE32), ("bf16", 500, 72, 2600, forms.TILE64),
           ("bf16", 1000, 203, 4400, forms.TILE128), ("bf16", 200, 128, 64000, forms.TILE256),
           ("mxfp4", 60, 64, 90, forms.SPLIT), ("e2m1", 500, 96, 4400, forms.TILE64), ("mxfp4", 1000, 160, 1200, forms.TILE32)]


def _bank(g, fmt, P, n, k):
    """Matrices of whole numbers and the bank: bf16, or codes with a scale of 1."""
    if fmt == "bf16":
        w = _values(g, (P, n, k), True)
        return m.make_bank(m.MOE_FMT_BF16, w), _f64(w)
    codes = g.choice(np.array([0, 2, 4, 10, 12]), (P, n, k))           # 0, 1, 2, -1, -2
    w = np.array([0.0, 0, 1, 0, 2, 0, 0, 0, 0, 0, -1, 0, -2])[codes]
    packed = torch.from_numpy((codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)).cuda()
    blk, one = (16, 0x38) if fmt == "e2m1" else (32, 127)
    scales = torch.full((P, n, k // blk), one, dtype=torch.uint8, device="cuda")
    return m.make_bank(m.MOE_FMT_E2M1 if fmt == "e2m1" else m.MOE_FMT_MXFP4, packed, scales), w


@pytest.mark.parametrize("case", CLIPPED, ids=lambda c: "-".join(str(v) for v in c[:4]) + "-" + forms.NAMES[c[4]])
def test_offsets_out_of_order_are_cut_to_the_range(case):
    """x and out lie in the middle of larger buffers.  Of the groups [40, 10), [10, past the end), [past the end,
    before the start) and [before the start, 20) the second and the last have places; 10 to 19 are named twice."""
    fmt, n, k, R, form = case
    print("clipped", *case, flush=True)
    g = W.rng(145, *case[:4])
    bank, w = _bank(g, fmt, 4, n, k)
    assert forms.form_of(fmt, n, k, R, groups=4) == form
    rows = _values(g, (R + 6, k), True)
    rows[:3], rows[R + 3:] = float("nan"), float("nan")
    big = torch.full((R + 6, n), 77.0, device="cuda")
    x, out = rows[3:R + 3], big[3:R + 3]
    m.moe_grouped_product(bank, x, _i32([40, 10, 2 ** 31 - 1, -2 ** 31, 20]), out)
    got, xs = _f64(out), _f64(x)
    assert (got[:10] == xs[:10] @ w[3].T).all() and (got[20:] == xs[20:] @ w[1].T).all()
    assert (big[:3] == 77).all() and (big[R + 3:] == 77).all()
    # all places named twice, by the first and by the third group: more pieces than a call has blocks
    big.fill_(77.0)
    m.moe_grouped_product(bank, x, _i32([0, R, 0, R + 5, 0]), out)
    got, e = _f64(out), (xs @ w[0].T, xs @ w[2].T)
    assert ((got == e[0]) | (got == e[1]) | (got == 77)).all()
    assert (big[:3] == 77).all() and (big[R + 3:] == 77).all()
