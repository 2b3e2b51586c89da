"""Sizes past the limits of the 4-bit rows and the MXFP4 products are
unsupported, not invalid (no GPU needed)."""
import ctypes as C

import pytest

import expert_slot_cache_moe_amd as m

P = 4096   # a plausible, aligned address; nothing reads it


@pytest.mark.parametrize("H,F,status", [
    (64, (1 << 19) + 32, m.MOE_UNSUPPORTED), (64, 1 << 30, m.MOE_UNSUPPORTED), ((1 << 16) + 32, 64, m.MOE_UNSUPPORTED),
    (64, (1 << 16) + 32, m.MOE_UNSUPPORTED), (64, 0, m.MOE_INVALID_ARG), (64, -32, m.MOE_INVALID_ARG),
    (0, 64, m.MOE_INVALID_ARG),
])
def test_routed_mx_sizes_past_its_limits(H, F, status):
    pool = m.moe_pool_t()
    pool.weight_format, pool.num_rows, pool.hidden, pool.ffn = m.MOE_FMT_MXFP4, 4, H, F
    for b in range(4):
        pool.banks_dev[b] = P
    assert m.lib().moe_routed_decode_mx(C.byref(pool), P, P, P, 2, 2, None, P, P, 1 << 50, None) == status
    assert m.moe_routed_mx_workspace_bytes(4, H, F, 2, 2) == 0


@pytest.mark.parametrize("fmt", [m.MOE_FMT_E2M1, m.MOE_FMT_MXFP4])
@pytest.mark.parametrize("rows,cols", [((1 << 32) + 1, 32), (4, (1 << 19) + 32)])
def test_rows_past_their_limits(fmt, rows, cols):
    assert m.lib().moe_quantize_rows(fmt, 1, P, cols, rows, cols, None, 0, P, P, None) == m.MOE_UNSUPPORTED
    assert m.lib().moe_dequantize_rows(fmt, P, P, rows, cols, None, 0, 1, P, cols, None) == m.MOE_UNSUPPORTED
