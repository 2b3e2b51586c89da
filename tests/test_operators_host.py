"""Refusals of the scored router, the 4-bit rows and the MXFP4 products:
every bad argument is an error status before anything is launched (no GPU
needed); workspace sizes; the plain 64-bit forms on worked values."""
import ctypes as C

import numpy as np
import pytest

import expert_slot_cache_moe_amd as m
import operator_ref as ref

P = 4096   # a plausible, aligned address; nothing reads it


def _status(fn, *args):
    return getattr(m.lib(), fn)(*args)


def _router(**kw):
    r = m.make_router(**{k: v for k, v in kw.items() if k != "bias_dev"})
    r.bias_dev = kw.get("bias_dev")
    return r


def _route(router=None, type=0, logits=P, stride=256, T=4, E=256, K=8, ids=P, w=P):
    r = _router() if router is None else router
    return _status("moe_route", C.byref(r) if r else None, type, logits, stride, T, E, K, ids, w, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(E=0, K=1), 1), (dict(K=0), 1), (dict(K=65), 1), (dict(E=4, K=5), 1),
    (dict(stride=255), 1), (dict(type=2), 1), (dict(type=-1), 1), (dict(logits=None), 1), (dict(ids=None), 1),
    (dict(w=None), 1), (dict(logits=P + 2), 1), (dict(type=1, logits=P + 1), 1), (dict(ids=P + 2), 1),
    (dict(E=2049, stride=2049), 2), (dict(T=(1 << 24) + 1), 2), (dict(router=_router(score=2)), 1),
    (dict(router=_router(num_groups=7)), 1), (dict(router=_router(num_groups=0)), 1),
    (dict(router=_router(num_groups=8, top_groups=9)), 1), (dict(router=_router(num_groups=8, top_groups=0)), 1),
    (dict(router=_router(num_groups=128, top_groups=2)), 2), (dict(router=_router(group_score=2)), 1),
    (dict(router=_router(renormalize=2)), 1), (dict(router=_router(scale=float("nan"))), 1),
    (dict(router=_router(scale=float("inf"))), 1), (dict(router=_router(bias_dev=P + 1)), 1), (dict(router=0), 1),
])
def test_route_refuses(kw, status):
    assert _route(**kw) == status
    assert m.moe_last_error()


def test_route_of_no_rows_is_fine():
    assert _route(T=0, logits=None, ids=None, w=None) == 0


def _rows(fn="moe_quantize_rows", fmt=2, type=1, dense=P, stride=64, rows=4, cols=64, glob=None, per=0,
          codes=P, scales=P):
    if fn == "moe_quantize_rows":
        return _status(fn, fmt, type, dense, stride, rows, cols, glob, per, codes, scales, None)
    return _status(fn, fmt, codes, scales, rows, cols, glob, per, type, dense, stride, None)


@pytest.mark.parametrize("fn", ["moe_quantize_rows", "moe_dequantize_rows"])
@pytest.mark.parametrize("kw,status", [
    (dict(fmt=0), 1), (dict(fmt=3), 1), (dict(type=2), 1), (dict(rows=-1), 1), (dict(cols=0), 1),
    (dict(cols=48), 1), (dict(fmt=1, cols=24), 1), (dict(stride=63), 1), (dict(glob=P, per=1), 1),
    (dict(fmt=1, glob=P, per=0), 1), (dict(fmt=1, glob=P + 2, per=1), 1), (dict(dense=None), 1),
    (dict(codes=None), 1), (dict(scales=None), 1), (dict(codes=P + 8), 1), (dict(fmt=1, codes=P + 4), 1),
    (dict(dense=P + 1), 1), (dict(type=0, dense=P + 2), 1), (dict(rows=(1 << 32) + 1), 2),
    (dict(cols=1 << 20, stride=1 << 20), 2),
])
def test_rows_refuse(fn, kw, status):
    assert _rows(fn, **kw) == status
    assert m.moe_last_error()


@pytest.mark.parametrize("fn", ["moe_quantize_rows", "moe_dequantize_rows"])
def test_no_rows_are_fine(fn):
    assert _rows(fn, rows=0, dense=None, codes=None, scales=None) == 0


def _bank(num_rows=4, n=32, k=64, codes=P, scales=P):
    b = m.moe_mx_bank_t()
    b.num_rows, b.n, b.k, b.codes_dev, b.scales_dev = num_rows, n, k, codes, scales
    return b


def _product(bank=None, x=P, stride=64, idx=P, T=2, K=2, swiglu=0, type=1, out=P, ws=P, ws_bytes=1 << 30):
    b = _bank() if bank is None else bank
    return _status("moe_mx_product", C.byref(b) if b else None, x, stride, idx, T, K, swiglu, type, out, ws,
                   ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(bank=0), 1), (dict(bank=_bank(num_rows=0)), 1), (dict(bank=_bank(n=0)), 1), (dict(bank=_bank(k=48)), 1),
    (dict(bank=_bank(k=0)), 1), (dict(bank=_bank(num_rows=32769)), 2), (dict(bank=_bank(n=(1 << 20) + 1)), 2),
    (dict(bank=_bank(k=(1 << 16) + 32)), 2), (dict(bank=_bank(codes=None)), 1), (dict(bank=_bank(scales=None)), 1),
    (dict(bank=_bank(codes=P + 8)), 1), (dict(T=-1), 1), (dict(K=0), 1), (dict(K=65), 2),
    (dict(T=131072, K=2), 2), (dict(swiglu=2), 1), (dict(bank=_bank(n=33), swiglu=1), 1), (dict(type=3), 1),
    (dict(stride=63), 1), (dict(idx=None), 1), (dict(idx=None, K=1), 1), (dict(x=None), 1), (dict(out=None), 1),
    (dict(ws=None), 1), (dict(x=P + 1), 1), (dict(out=P + 1), 1), (dict(type=0, out=P + 2), 1),
    (dict(idx=P + 2), 1), (dict(ws=P + 128), 1), (dict(ws_bytes=16), 1),
    # 40961 runs of 16384 blocks, 33281 of 2048: 2^32 threads and more
    (dict(bank=_bank(num_rows=32768, n=1 << 20, k=32), T=65536), 2),
    (dict(bank=_bank(num_rows=32768, n=1 << 18, k=4096), stride=4096, T=16384), 2),
])
def test_product_refuses(kw, status):
    assert _product(**kw) == status
    assert m.moe_last_error()


def test_product_of_no_rows_is_fine():
    assert _product(T=0, x=None, out=None, ws=None) == 0


def _pool(fmt=2, rows=4, H=64, F=32, bank=P):
    p = m.moe_pool_t()
    p.weight_format, p.num_rows, p.hidden, p.ffn = fmt, rows, H, F
    for b in range(6):
        p.banks_dev[b] = bank
    return p


def _routed(pool=None, x=P, idx=P, w=P, T=2, K=2, add=None, out=P, ws=P, ws_bytes=1 << 30):
    b = _pool() if pool is None else pool
    return _status("moe_routed_decode_mx", C.byref(b) if b else None, x, idx, w, T, K, add, out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(pool=0), 1), (dict(pool=_pool(fmt=0)), 1), (dict(pool=_pool(fmt=1)), 1), (dict(pool=_pool(rows=0)), 1),
    (dict(pool=_pool(H=48)), 2), (dict(pool=_pool(F=48)), 2), (dict(pool=_pool(bank=None)), 1),
    (dict(pool=_pool(bank=P + 8)), 1), (dict(T=-1), 1), (dict(K=0), 1), (dict(T=65536, K=1), 2), (dict(x=None), 1),
    (dict(x=P + 8), 1), (dict(idx=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(ws=P + 64), 1), (dict(ws_bytes=100), 1), (dict(add=P + 2), 1), (dict(out=P + 1), 1),
    (dict(pool=_pool(rows=32768, H=32, F=1 << 18), T=32768, ws_bytes=1 << 50), 2),
    (dict(pool=_pool(rows=32768, H=1 << 16, F=4096), T=65535, ws_bytes=1 << 50), 2),
])
def test_routed_mx_refuses(kw, status):
    assert _routed(**kw) == status
    assert m.moe_last_error()


def test_workspace_sizes():
    assert m.moe_mx_product_workspace_bytes(4, 32, 48, 1, 1) == 0
    assert m.moe_mx_product_workspace_bytes(4, 32, 64, 1 << 17, 2) == 0
    small = m.moe_mx_product_workspace_bytes(4, 32, 64, 1, 2)
    # the quantised rows alone are T (k/2 + k/32) bytes, the sorted routes 4 T K
    T, K, k = 1000, 4, 4096
    big = m.moe_mx_product_workspace_bytes(256, 2048, k, T, K)
    assert 0 < small < big and big >= T * (k // 2 + k // 32) + 4 * T * K
    assert m.moe_routed_mx_workspace_bytes(4, 64, 48, 1, 1) == 0
    H, F = 1024, 256
    assert m.moe_routed_mx_workspace_bytes(160, H, F, 600, 2) >= 1200 * (2 * F + 4 * H)


def test_layer_step_with_a_null_cache_is_refused():
    r = _router()
    assert _status("moe_layer_decode_router", None, 0, P, P, 1, 2, C.byref(r), None, -1, P, None, None, None) == 1


def test_hybrid_step_refuses_a_router():
    # the host threads' half routes by the plain top-k: a router must not be dropped in silence
    from expert_slot_cache_moe_amd.layer import SlotCacheLayers

    lay = object.__new__(SlotCacheLayers)
    lay.routers = [None, _router(score=m.MOE_SCORE_SIGMOID)]
    with pytest.raises(ValueError, match="router"):
        lay.decode_hybrid(0, None, None, 2, None)


# ---------------------------------------------------------------- the plain forms

def test_plain_route_on_worked_rows():
    ln = np.log
    # softmax scores 0.5, 0.3, 0.2; a bias lifts the last over the second
    l = ln(np.array([[0.5, 0.3, 0.2]]))
    ids, w = ref.route(l, 2, score="softmax")
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[0.625, 0.375]])
    ids, w = ref.route(l, 2, score="softmax", renorm=False, scale=2.0, bias=np.array([0, 0, 0.2]))
    assert ids.tolist() == [[0, 2]] and np.allclose(w, [[1.0, 0.4]])
    # groups of two: maxima 3, 4 keep the second; sums of the two best keep the first
    g = np.array([[3.0, 3.0, 4.0, -9.0]])
    assert ref.route(g, 1, score="sigmoid", groups=2, top_groups=1)[0].tolist() == [[2]]
    assert ref.route(g, 1, score="sigmoid", groups=2, top_groups=1, top2=True)[0].tolist() == [[0]]
    # masked experts are never picked; what is missing is -1 with weight 0
    ids, w = ref.route(np.array([[-np.inf, 1.0, np.nan], [-np.inf] * 3]), 2, score="softmax")
    assert ids.tolist() == [[1, -1], [-1, -1]] and np.allclose(w, [[1, 0], [0, 0]])


def test_plain_rows_on_worked_values():
    # largest 6: scale 1; middles go to the even code
    x = np.zeros((1, 32))
    x[0, :9] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.26]
    codes, sc, vals = ref.quantize(x, "mxfp4")
    assert sc.tolist() == [[127]]
    assert vals[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -0.5]
    assert codes[0, 0] == 7 and codes[0, 4] == 9
    assert (ref.decode_mxfp4(codes, sc) == vals).all()
    # largest 7.9 saturates at 6; nothing at all gives the smallest scale
    x[0, 0] = 7.9
    assert ref.quantize(x, "mxfp4")[2][0, 0] == 6
    assert ref.quantize(np.zeros((1, 32)), "mxfp4")[1].tolist() == [[0]]
    # E2M1: 12 / 6 = 2 = E4M3 0x40; codes of x / 2
    y = np.zeros((1, 16))
    y[0, :3] = [12.0, 1.0, -3.0]
    codes, sc, vals = ref.quantize(y, "e2m1")
    assert sc.tolist() == [[0x40]] and vals[0, :3].tolist() == [12, 1, -3]
    assert ref.quantize(y, "e2m1", glob=[2.0], per=1)[1].tolist() == [[0x38]]
    y[0, 0] = np.nan
    assert ref.quantize(y, "e2m1")[1].tolist() == [[0x7F]] and np.isnan(ref.quantize(y, "e2m1")[2]).all()


def test_plain_product_is_the_matrix_product():
    g = np.random.default_rng(3)
    codes = g.integers(0, 256, (2, 3, 32), dtype=np.uint8)
    scales = g.integers(120, 130, (2, 3, 2), dtype=np.uint8)
    x = g.standard_normal((2, 64))
    idx = np.array([[1, -1], [0, 1]])
    y, a = ref.product(codes, scales, x, idx)
    w = ref.decode_mxfp4(codes, scales)
    assert np.allclose(y, [w[1] @ x[0], np.zeros(3), w[0] @ x[1], w[1] @ x[1]]) and (a >= np.abs(y) - 1e-12).all()
