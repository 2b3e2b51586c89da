"""SlotCacheLayers.prefill checks all its arguments before its first call into
the library.  No GPU: the calls are recorded instead, on tensors in host
memory."""
import pytest
import torch

import expert_slot_cache_moe_amd as m
from expert_slot_cache_moe_amd import layer as layer_module
from expert_slot_cache_moe_amd.layer import SlotCacheLayers

L, E, H, F, K, T = 2, 12, 64, 32, 3, 9
BF16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """What prefill has called, by name."""
    made = []
    monkeypatch.setattr(layer_module, "_on_current_device", lambda *t: m._load_torch())
    for name in ("moe_topk", "moe_route", "moe_shared_prefill", "moe_routed_prefill"):
        monkeypatch.setattr(layer_module, name, lambda *a, _name=name, **kw: made.append(_name))
    return made


def _pool(**kw):
    p = m.moe_pool_t()
    p.weight_format, p.hidden, p.ffn, p.num_rows = m.MOE_FMT_BF16, H, F, E
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.fixture
def layers():
    lay = SlotCacheLayers.__new__(SlotCacheLayers)
    lay.L, lay.E, lay.H, lay.F, lay.fmt, lay.device, lay.cache = L, E, H, F, m.MOE_FMT_BF16, torch.device("cpu"), None
    lay.routers = [None, m.moe_router_t()]
    shared = m.moe_shared_t()
    shared.ffn = F
    lay.shared = [shared, None]
    return lay


def _args(**kw):
    a = dict(x=torch.zeros((T, H), dtype=BF16), logits=torch.zeros((T, E)), K=K, out=torch.zeros((T, H), dtype=BF16),
             ids_out=torch.zeros((T, K), dtype=torch.int32), w_out=torch.zeros((T, K)), pool=_pool())
    a.update(kw)
    return a


def test_a_good_call_reaches_the_library(calls, layers):
    layers.prefill(0, **_args())
    assert calls == ["moe_topk", "moe_shared_prefill", "moe_routed_prefill"]
    calls.clear()
    layers.prefill(1, **_args(logits=torch.zeros((T, E + 3))[:, :E], ids_out=None, w_out=None))
    assert calls == ["moe_route", "moe_routed_prefill"]
    calls.clear()
    # a pool in another format, of other widths and rows
    layers.prefill(1, **_args(pool=_pool(weight_format=m.MOE_FMT_MXFP4, ffn=4 * F, num_rows=3)))
    assert calls == ["moe_route", "moe_routed_prefill"]


MANY = 65536
BAD = {
    "x in fp32": dict(x=torch.zeros((T, H))),
    "x of other rows": dict(x=torch.zeros((T - 1, H), dtype=BF16)),
    "x of other columns": dict(x=torch.zeros((T, H + 1), dtype=BF16)),
    "rows of x apart": dict(x=torch.zeros((T, H + 2), dtype=BF16)[:, :H]),
    "out in fp32": dict(out=torch.zeros((T, H))),
    "rows of out apart": dict(out=torch.zeros((T, H + 2), dtype=BF16)[:, :H]),
    "logits in bf16": dict(logits=torch.zeros((T, E), dtype=BF16)),
    "logits of other experts": dict(logits=torch.zeros((T, E - 1))),
    "columns of logits apart": dict(logits=torch.zeros((E, T)).t()),
    "ids in int64": dict(ids_out=torch.zeros((T, K), dtype=torch.int64)),
    "rows of ids apart": dict(ids_out=torch.zeros((T, K + 1), dtype=torch.int32)[:, :K]),
    "one row of ids for all": dict(ids_out=torch.zeros((1, K), dtype=torch.int32).expand(T, K)),
    "rows of w apart": dict(w_out=torch.zeros((T, K + 1))[:, :K]),
    "another K": dict(K=K + 1),
    "no K": dict(K=0, ids_out=None, w_out=None),
    "too large a K": dict(K=65, ids_out=None, w_out=None),
    "too many tokens": dict(x=torch.zeros((MANY, H), dtype=BF16), logits=torch.zeros((MANY, E)),
                            out=torch.zeros((MANY, H), dtype=BF16), ids_out=None, w_out=None),
    "a pool without columns": dict(pool=_pool(ffn=0)),
    "a pool of another hidden": dict(pool=_pool(hidden=2 * H)),
    "a pool of no format": dict(pool=_pool(weight_format=9)),
    "a pool without rows": dict(pool=_pool(num_rows=0)),
}


@pytest.mark.parametrize("layer", range(L))
@pytest.mark.parametrize("case", BAD)
def test_a_bad_call_is_refused_before_anything_is_called(calls, layers, layer, case):
    with pytest.raises((ValueError, m.MoeError)):
        layers.prefill(layer, **_args(**BAD[case]))
    assert calls == []


@pytest.mark.parametrize("layer", [-1, L])
def test_no_such_layer(calls, layers, layer):
    with pytest.raises(ValueError):
        layers.prefill(layer, **_args())
    assert calls == []


def test_strided_logits_need_a_router(calls, layers):
    with pytest.raises(ValueError):
        layers.prefill(0, **_args(logits=torch.zeros((T, E + 3))[:, :E]))
    assert calls == []
