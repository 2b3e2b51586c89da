"""The activations' values over their whole range, relative to the value, in
every form of the products (activation_ref.py, where the bounds are derived).
x is zero, so that each column is the activation of its bias."""
import numpy as np
import pytest
import torch

import activation_ref as ref
import expert_slot_cache_moe_amd as m
import product_forms as forms
from expert_slot_cache_moe_amd import workloads as W
from product_ref import HALF, TINY

pytestmark = pytest.mark.gpu

ACT = {"silu": m.MOE_ACT_SILU, "gelu": m.MOE_ACT_GELU, "swiglu": m.MOE_ACT_SWIGLU}


def _arguments(n):
    """Both signs, from 0 to past the point where each function is below fp32's range, and far beyond."""
    ends = np.array([0.0, -0.0, 1e-38, -1e-38, 1e-20, -1e-20, 13.0, -13.0, -13.2, -13.4, 14.0, -14.0, -20.0, 87.0, -87.0,
                     -88.5, 89.0, -89.0, -104.0, 200.0, -200.0, 1e10, -1e10, 1e19, -1e19, 3e38, -3e38], np.float32)
    rest = n - len(ends)
    return np.concatenate([ends, np.linspace(-14, 14, rest - rest // 2, dtype=np.float32),
                           np.linspace(-90, 3, rest // 2, dtype=np.float32)])


# rows, n (k is 64) and the form that they take
SIZES = [(2, 1000, forms.SPLIT), (1100, 1500, forms.TILE32), (4100, 500, forms.TILE64), (8200, 500, forms.TILE128),
         (65600, 200, forms.TILE256)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
@pytest.mark.parametrize("T,n,form", SIZES, ids=lambda v: str(v))
def test_activations_are_near_relative_to_their_values(T, n, form, act, dtype):
    k, glu = 64, act == "swiglu"
    cols = n // 2 if glu else n
    print("activation", act, T, n, dtype, flush=True)
    assert forms.form_of("bf16", n, k, T, swiglu=glu) == form
    y = _arguments(n)
    if glu:
        y[cols:] = np.resize(np.array([1.0, -3.5, 1e-3], np.float32), cols)
        y[:cols] = _arguments(cols)
        y[:cols][np.abs(y[:cols]) > 1e37] = 5.0            # times 3.5 past fp32
    g = W.rng(130, act, T)
    w = torch.from_numpy(W.normal_bf16(g, (1, n, k)).view(np.int16)).cuda().view(torch.bfloat16)
    out = torch.full((T, cols), 77.0, dtype=dtype, device="cuda")
    m.moe_linear(m.make_bank(m.MOE_FMT_BF16, w), torch.zeros((T, k), dtype=torch.bfloat16, device="cuda"), out,
                 bias=torch.from_numpy(y).cuda(), activation=ACT[act])
    assert (out == out[0]).all()
    got, y = out[0].double().cpu().numpy(), y.astype(np.float64)[None]
    val, bnd = ref.activate(y, 0 * y, act)
    name = str(dtype).split(".")[1]
    # (past bf16's largest: infinity)
    fin = np.isfinite(got)
    assert (np.abs(val[0][~fin]) > 3.38e38).all()
    excess = np.abs(got - val[0])[fin] - (bnd[0] * (1 + HALF[name]) + np.abs(val[0]) * HALF[name] + TINY[name])[fin]
    worst = int(np.argmax(excess))
    assert excess[worst] <= 0, (y[0][:cols][fin][worst], got[fin][worst], val[0][fin][worst])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [2, 4100])
def test_activations_of_infinities_and_nan(act, T):
    """By their formulas: y / (1 + exp(-y)) and y (1 + erf) / 2 of minus infinity are infinity over infinity, infinity
    times 0."""
    n, k = 512, 64
    v = np.array([np.inf, -np.inf, np.nan, 1.0], np.float32)
    w = torch.zeros((1, n, k), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((T, n), device="cuda")
    m.moe_linear(m.make_bank(m.MOE_FMT_BF16, w), torch.zeros((T, k), dtype=torch.bfloat16, device="cuda"), out,
                 bias=torch.from_numpy(np.resize(v, n)).cuda(), activation=ACT[act])
    got = out.cpu().numpy().reshape(T, n // 4, 4)
    assert (got[..., 0] == np.inf).all() and np.isnan(got[..., 1:3]).all() and np.isfinite(got[..., 3]).all()
