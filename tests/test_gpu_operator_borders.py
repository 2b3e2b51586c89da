"""Borders of the 4-bit rows on the GPU, against the plain 64-bit forms
(operator_ref.py): codes and scales are equal."""
import numpy as np
import pytest
import torch

import expert_slot_cache_moe_amd as m
import operator_ref as ref
from expert_slot_cache_moe_amd import workloads as W

pytestmark = pytest.mark.gpu


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
