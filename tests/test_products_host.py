"""Refusals of the route lists, the grouped and dense products and the routed
experts of a prompt: every bad argument is an error status before anything is
launched (no GPU needed); workspace sizes; the plain forms on worked values."""
import ctypes as C

import numpy as np
import pytest

import expert_slot_cache_moe_amd as m
import product_ref as ref

P = 4096   # a plausible, aligned address; nothing reads it


def _bank(fmt=0, num_rows=4, n=32, k=64, w=P, scales=None, glob=None):
    b = m.moe_bank_t()
    b.weight_format, b.num_rows, b.n, b.k = fmt, num_rows, n, k
    b.weights_dev, b.scales_dev, b.globals_dev = w, P if scales is None and fmt else scales or None, glob
    return b


def _lists(idx=P, T=4, K=2, rows=8, offsets=P, order=P, ws=None, ws_bytes=0):
    return m.lib().moe_group_routes(idx, T, K, rows, offsets, order, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(K=0), 1), (dict(rows=0), 1), (dict(rows=-3), 1), (dict(rows=32769), 2),
    (dict(T=1 << 22, K=2), 2), (dict(idx=None), 1), (dict(offsets=None), 1), (dict(order=None), 1),
    (dict(idx=P + 2), 1), (dict(offsets=P + 1), 1), (dict(order=P + 2), 1), (dict(T=1 << 16), 1),
    (dict(T=1 << 16, ws=P, ws_bytes=64), 1), (dict(T=1 << 16, ws=P + 2, ws_bytes=1 << 30), 1),
    (dict(T=1 << 16, ws=None, ws_bytes=1 << 30), 1), (dict(offsets=None, T=0), 1),
])
def test_lists_refuse(kw, status):
    assert _lists(**kw) == status
    assert m.moe_last_error()


def _grouped(bank=None, x=P, x_stride=64, x_rows=8, offsets=P, G=4, mats=None, gather=None, div=1, scatter=None,
             R=8, act=0, bias_type=0, bias=None, out_type=1, out=P, out_stride=32, out_rows=8):
    b = _bank() if bank is None else bank
    return m.lib().moe_grouped_product(C.byref(b) if b else None, x, x_stride, x_rows, offsets, G, mats, gather, div,
                                       scatter, R, act, bias_type, bias, out_type, out, out_stride, out_rows, None)


def _linear(bank=None, x=P, x_stride=64, T=8, act=0, bias_type=0, bias=None, res_type=1, res=None, res_stride=32,
            out_type=1, out=P, out_stride=32):
    b = _bank(num_rows=1) if bank is None else bank
    return m.lib().moe_linear(C.byref(b) if b else None, x, x_stride, T, act, bias_type, bias, res_type, res,
                              res_stride, out_type, out, out_stride, None)


SHARED = [
    (dict(bank=0), 1), (dict(bank=_bank(fmt=3)), 1), (dict(bank=_bank(fmt=-1)), 1), (dict(bank=_bank(num_rows=0)), 1),
    (dict(bank=_bank(n=0)), 1), (dict(bank=_bank(k=0)), 1), (dict(bank=_bank(fmt=1, k=48)), 1),
    (dict(bank=_bank(fmt=2, k=16), x_stride=64), 1), (dict(bank=_bank(num_rows=32769)), 2),
    (dict(bank=_bank(n=(1 << 20) + 1)), 2), (dict(bank=_bank(k=(1 << 16) + 1)), 2), (dict(bank=_bank(w=None)), 1),
    (dict(bank=_bank(w=P + 1)), 1), (dict(bank=_bank(fmt=1, w=P + 8)), 1), (dict(bank=_bank(fmt=1, scales=0)), 1),
    (dict(bank=_bank(fmt=1, scales=P + 1)), 1), (dict(bank=_bank(fmt=1, glob=P + 2)), 1),
    (dict(bank=_bank(fmt=2, glob=P)), 1), (dict(bank=_bank(fmt=0, glob=P)), 1), (dict(act=4), 1), (dict(act=-1), 1),
    (dict(out_type=2), 1), (dict(bias=P, bias_type=2), 1), (dict(bias=P + 2), 1), (dict(bias=P + 1, bias_type=1), 1),
    (dict(x_stride=63), 1), (dict(out_stride=31), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(x=P + 1), 1),
    (dict(out=P + 1), 1), (dict(out=P + 2, out_type=0), 1),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(bank=_bank(n=33), act=3), 1), (dict(R=-1), 1), (dict(R=(1 << 22) + 1), 2), (dict(G=0), 1),
    (dict(G=32769, mats=P), 2), (dict(G=5), 1), (dict(offsets=None), 1), (dict(gather=P, div=0), 1),
    (dict(x_rows=7), 1), (dict(x_rows=0, gather=P), 1), (dict(out_rows=7), 1), (dict(out_rows=-1, scatter=P), 1),
    (dict(offsets=P + 2), 1), (dict(mats=P + 1), 1), (dict(gather=P + 2), 1), (dict(scatter=P + 2), 1),
    # 2^20 columns for 2^22 places: 2^32 threads and more
    (dict(bank=_bank(n=1 << 20, k=1), R=1 << 22, x_rows=1 << 22, out_rows=1 << 22, out_stride=1 << 20), 2),
])
def test_grouped_product_refuses(kw, status):
    assert _grouped(**kw) == status
    assert m.moe_last_error()


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(bank=_bank(num_rows=1, n=33), act=3), 1), (dict(T=-1), 1), (dict(T=(1 << 22) + 1), 2), (dict(bank=_bank()), 1),
    (dict(res=P, res_type=2), 1), (dict(res=P, res_stride=31), 1), (dict(res=P + 1), 1), (dict(res=P + 2, res_type=0), 1),
])
def test_linear_refuses(kw, status):
    assert _linear(**kw) == status
    assert m.moe_last_error()


def test_no_rows_are_fine():
    assert _grouped(R=0, x=None, out=None, x_rows=0, out_rows=0) == 0
    assert _linear(T=0, x=None, out=None) == 0


def _pool(fmt=0, rows=4, H=64, F=32, bank=P):
    p = m.moe_pool_t()
    p.weight_format, p.num_rows, p.hidden, p.ffn = fmt, rows, H, F
    for b in range(m.MOE_MAX_BANKS):
        p.banks_dev[b] = bank
    return p


def _prefill(pool=None, x=P, idx=P, w=P, T=4, K=2, addend=None, out=P, ws=P, ws_bytes=1 << 30):
    p = _pool() if pool is None else pool
    return m.lib().moe_routed_prefill(C.byref(p) if p else None, x, idx, w, T, K, addend, out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(pool=0), 1), (dict(pool=_pool(fmt=3)), 1), (dict(pool=_pool(rows=0)), 1), (dict(pool=_pool(rows=32769)), 2),
    (dict(pool=_pool(H=0)), 1), (dict(pool=_pool(F=-1)), 1), (dict(pool=_pool(fmt=1, H=48)), 2),
    (dict(pool=_pool(fmt=2, F=16)), 2), (dict(pool=_pool(H=(1 << 16) + 32)), 2), (dict(pool=_pool(bank=None)), 1),
    (dict(pool=_pool(fmt=1, bank=P + 8)), 1), (dict(T=-1), 1), (dict(T=65536), 2), (dict(K=0), 1), (dict(K=65), 2),
    (dict(x=None), 1), (dict(idx=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(x=P + 1), 1), (dict(idx=P + 2), 1), (dict(w=P + 2), 1), (dict(addend=P + 2), 1), (dict(out=P + 1), 1),
    (dict(ws=P + 64), 1), (dict(ws_bytes=256), 1),
])
def test_prefill_refuses(kw, status):
    assert _prefill(**kw) == status
    assert m.moe_last_error()


def test_prefill_of_no_tokens_is_fine():
    assert _prefill(T=0, x=None, idx=None, w=None, out=None, ws=None) == 0


def test_workspace_sizes():
    assert m.moe_group_routes_workspace_bytes(256, 1, 8) == 0
    assert m.moe_group_routes_workspace_bytes(512, 16384, 10) > 0
    assert m.moe_group_routes_workspace_bytes(0, 1, 8) == 0
    assert m.moe_group_routes_workspace_bytes(32769, 16384, 10) == 0
    got = m.moe_routed_prefill_workspace_bytes(m.MOE_FMT_BF16, 256, 4096, 1024, 4096, 6)
    assert got >= 24576 * (4 + 2 * 1024 + 4 * 4096) + 257 * 4
    assert m.moe_routed_prefill_workspace_bytes(m.MOE_FMT_E2M1, 256, 48, 32, 4, 2) == 0


def test_plain_lists_of_a_worked_example():
    offsets, order = ref.lists([[2, 0], [-1, 2], [0, 7], [2, 1]], 3)
    assert offsets.tolist() == [0, 2, 3, 6]
    assert order.tolist() == [1, 4, 7, 0, 3, 6, 2, 5]


def test_plain_product_of_a_worked_example():
    w = np.array([[[1.0, 2.0], [3.0, -1.0]], [[0.5, 0.5], [0.0, 4.0]]])
    x = np.array([[1.0, 1.0], [2.0, 0.0], [0.0, -1.0]])
    # places 0 and 1 in group 0, place 2 in group 1; matrices swapped; results scattered
    done, v, _ = ref.grouped(w, x, [0, 2, 3], 5, matrices=[1, 0], scatter=[4, 0, 2], bias=np.array([[1, 0], [0, 2.0]]))
    assert done.tolist() == [True, False, True, False, True]
    assert v[4].tolist() == [1.0, 6.0] and v[0].tolist() == [1.0, 2.0] and v[2].tolist() == [-1.0, 1.0]
    y, _ = ref.product(np.array([[0.0, 1.0], [2.0, 0.0]]), np.array([[3.0, 1.0]]), "swiglu")
    assert np.allclose(y, 6 / (1 + np.exp(-1.0)))
