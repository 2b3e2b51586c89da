"""Borders of the scored router, the 4-bit rows and the layer's 4-bit banks
on the GPU, against the plain 64-bit forms (operator_ref.py).  Ids, codes,
scales and bf16 values are equal; routing weights are 64-bit arithmetic
rounded once to fp32 (2^-24, and the difference of two 64-bit exponentials)."""
import numpy as np
import pytest
import torch

import expert_slot_cache_moe_amd as m
import operator_ref as ref
from expert_slot_cache_moe_amd import workloads as W

pytestmark = pytest.mark.gpu

LOW = float(np.finfo(np.float32).min)


def _say(*a):
    print(*a, flush=True)


def _f64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------- E2M1 rows far past the largest scale

def _check_e2m1(x, glob):
    """One global scale to a row: codes and scales equal to the plain form's."""
    R, C = x.shape
    codes = torch.full((R, C // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, C // 16), 0xCD, dtype=torch.uint8, device="cuda")
    m.moe_quantize_rows(m.MOE_FMT_E2M1, x, codes, scales, globals=glob, rows_per_global=1)
    e_codes, e_scales, _ = ref.quantize(_f64(x), "e2m1", _f64(glob), 1)
    assert (scales.cpu().numpy() == e_scales).all()
    bad = codes.cpu().numpy() != e_codes
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_saturated_e2m1_blocks_take_the_largest_code_and_the_sign(dtype):
    # x / (448 g) of 2^-2 to 2^100 in one block, both signs; the reciprocal of 448 g is rounded up
    # to 16 bits or fewer in one global scale of some 500
    _say("saturated rows", dtype)
    g = W.rng(81, "saturated", str(dtype))
    globs = [np.float32(1 / 7) * np.float32(2.0) ** -j for j in range(20, 81)]
    globs += list(((g.random(6000) + 1) * 2.0 ** g.integers(-80, -20, 6000)).astype(np.float32))
    globs = np.array(globs, np.float32)
    x = np.zeros((len(globs), 128), np.float64)
    u = 448 * globs.astype(np.float64)
    x[:, 0] = np.minimum(u * 2.0 ** 100, 3e38)
    for j in range(1, 128):
        x[:, j] = u * 2.0 ** (j % 16 * 6.5 + g.random(len(globs)) - 2) * g.choice([-1.0, 1.0], len(globs))
    x[:, ::16] = np.minimum(u * 2.0 ** 60, 3e38)[:, None] * g.choice([-1.0, 1.0], (len(globs), 8))
    x = np.clip(x, -3e38, 3e38)
    _check_e2m1(torch.from_numpy(x.astype(np.float32)).to(dtype).cuda(), torch.from_numpy(globs).cuda())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_e2m1_quotients_below_the_smallest_float_are_zeros_of_the_sign(dtype):
    # blocks of one large value beside values down to the smallest: x / (s g) of 2^-149 and less
    _say("vanishing quotients", dtype)
    g = W.rng(85, "vanishing", str(dtype))
    R, C = 6000, 64
    globs = ((g.random(R) + 1) * 2.0 ** g.integers(20, 80, R)).astype(np.float32)
    x = (g.random((R, C)) + 1) * 2.0 ** g.integers(-133, -60, (R, C)) * g.choice([-1.0, 1.0], (R, C))
    x[:, ::16] = np.minimum(6 * globs[:, None].astype(np.float64) * 2.0 ** g.integers(-8, 9, (R, C // 16)), 3e38)
    _check_e2m1(torch.from_numpy(x.astype(np.float32)).to(dtype).cuda(), torch.from_numpy(globs).cuda())


# ---------------------------------------------------------------- two-best groups of lowest-value biases

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,K", [(16, 4, 2, 4), (64, 8, 3, 12), (160, 8, 5, 30), (1024, 16, 4, 64)])
@pytest.mark.parametrize("open_groups", [0, 1, 2])
def test_two_best_groups_whose_biases_sum_below_the_lowest_float(score, E, groups, top_groups, K, open_groups):
    # experts biased by the type's lowest value are available still: their groups fill the choice
    _say("lowest biases", score, E, groups, top_groups, K, open_groups)
    g = W.rng(82, "lowest", score, E, open_groups)
    T, gs = 9, E // groups
    x = g.standard_normal((T, E)).astype(np.float32)
    x[1] = 0.5
    x[2, ::3] = -np.inf
    for b in (np.full(E, LOW), np.where(g.random(E) < 0.3, LOW / 2, LOW), np.where(np.arange(E) % gs == 0, 0.0, LOW),
              np.where(np.arange(E) % gs < 2, -LOW, LOW)):
        b = b.astype(np.float32)
        b[:open_groups * gs] = 0.0
        router = m.make_router(score=m.MOE_SCORE_SIGMOID if score == "sigmoid" else m.MOE_SCORE_SOFTMAX,
                               num_groups=groups, top_groups=top_groups, group_score=m.MOE_GROUP_TOP2,
                               bias=torch.from_numpy(b).cuda())
        ids = torch.full((T, K), 77, dtype=torch.int32, device="cuda")
        w = torch.full((T, K), np.nan, dtype=torch.float32, device="cuda")
        m.moe_route(router, torch.from_numpy(x).cuda(), K, ids, w)
        e_ids, e_w = ref.route(x.astype(np.float64), K, score=score, groups=groups, top_groups=top_groups, top2=True,
                               bias=b.astype(np.float64))
        assert (ids.cpu().numpy() == e_ids).all()
        assert (np.abs(_f64(w) - e_w) <= np.abs(e_w) * (2.0 ** -24 + 1e-12) + 2.0 ** -150).all()


# ---------------------------------------------------------------- E2M1 values below the smallest normal number

def test_subnormal_e2m1_values_are_rounded_once_to_bf16():
    # products of a code value and a block scale that fp32 rounds onto the middle of two bf16 numbers
    _say("subnormal values")
    g = W.rng(83, "subnormal")
    grid = ref.e4m3_grid()
    globs, codes, scales = [], [], []
    for _ in range(4000):
        s = int(g.integers(1, 24))
        a = ref.VALUES[1:] * grid[s]
        # g near an odd multiple of 2^-134 over one of the values: the middles of bf16 below 2^-126
        v = a[g.integers(0, 7)]
        globs.append(np.float32((2 * int(g.integers(1, 128)) + 1) * 2.0 ** -134 / v))
        scales.append(s)
    globs = np.array(globs, np.float32)
    globs = np.where(g.random(4000) < 0.5, np.nextafter(globs, np.float32(1)), globs)
    R = len(globs)
    c = np.tile(np.arange(16, dtype=np.uint8), (R, 1))
    packed = torch.from_numpy(c[:, 0::2] | (c[:, 1::2] << 4)).cuda()
    out = torch.empty((R, 16), dtype=torch.bfloat16, device="cuda")
    m.moe_dequantize_rows(m.MOE_FMT_E2M1, packed, torch.from_numpy(np.array(scales, np.uint8))[:, None].cuda(), out,
                          globals=torch.from_numpy(globs).cuda(), rows_per_global=1)
    val = ref.VALUES[np.arange(16) & 7] * np.where(np.arange(16) & 8, -1.0, 1.0)
    v = val[None, :] * grid[np.array(scales)][:, None] * globs.astype(np.float64)[:, None]   # exact: at most 33 bits
    step = np.ldexp(1.0, np.maximum(np.frexp(np.where(v == 0, 1e-300, v))[1] - 8, -133))
    want = np.rint(v / step) * step                                                          # ties to even
    bad = _f64(out) != want
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), _f64(out)[bad][:4], want[bad][:4])


# ---------------------------------------------------------------- 4-bit banks of experts that are not finite

@pytest.mark.parametrize("fmt", ["mxfp4", "e2m1"])
def test_quantized_banks_keep_the_finite_blocks_beside_nan_and_infinity(fmt):
    from expert_slot_cache_moe_amd.layer import quantized_banks

    _say("banks", fmt)
    code = m.MOE_FMT_MXFP4 if fmt == "mxfp4" else m.MOE_FMT_E2M1
    E, H, F = 4, 64, 96
    g = W.rng(84, "banks", fmt)
    w13, w2 = W.bf16_expert_rows(g, E, H, F)
    w2.view(np.uint16)[1, 7] = 0x7F80             # +infinity
    w2.view(np.uint16)[2, 100] = 0x7FC0           # NaN
    w13.view(np.uint16)[0, 5] = 0xFF80            # -infinity
    w13.view(np.uint16)[3] = 0x7F80               # nothing else
    banks = [b.cpu().numpy() for b in quantized_banks(code, w13, w2, H, F)]
    per = 3 if fmt == "e2m1" else 2
    for i, (raw, n, k) in enumerate(((w13, 2 * F, H), (w2, H, F))):
        x = ref.bf16_f64(raw.view(np.uint16)).reshape(E * n, k)
        glob = None
        if fmt == "e2m1":
            glob = banks[per * i + 2].reshape(-1).view(np.float32)
            amax = np.where(np.isfinite(x), np.abs(x), 0.0).reshape(E, -1).max(1)
            assert np.allclose(glob, np.where(amax > 0, amax / 2688, 1.0), rtol=1e-6)
        codes, scales, vals = ref.quantize(x, fmt, glob, n)
        assert (banks[per * i].reshape(E * n, -1) == codes).all()
        assert (banks[per * i + 1].reshape(E * n, -1) == scales).all()
        assert np.isfinite(vals).any(1).reshape(E, n).all(1).sum() == E - (i == 0)
