"""The refusals of moe_shared_prefill: arguments are checked on the host, so
that no launch is reached and no device is needed."""
import ctypes as C

import pytest

import expert_slot_cache_moe_amd as m

P = 1 << 20      # stands for a device pointer; never followed


def _shared(ffn=64, w13=P, w2=P, gate=P):
    s = m.moe_shared_t()
    s.ffn, s.w13_dev, s.w2_dev, s.gate_dev = ffn, w13, w2, gate
    return s


def _call(shared=None, H=64, x=P, T=4, addend=P, ws=P, ws_bytes=1 << 30):
    s = _shared() if shared is None else shared
    return m.lib().moe_shared_prefill(C.byref(s) if s else None, H, x, T, addend, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(shared=0), 1), (dict(shared=_shared(ffn=0)), 1), (dict(shared=_shared(ffn=-4)), 1),
    (dict(shared=_shared(ffn=(1 << 16) + 1)), 2), (dict(shared=_shared(w13=None)), 1),
    (dict(shared=_shared(w2=None)), 1), (dict(shared=_shared(gate=None)), 1), (dict(shared=_shared(w13=P + 1)), 1),
    (dict(shared=_shared(w2=P + 1)), 1), (dict(shared=_shared(gate=P + 1)), 1), (dict(H=0), 1),
    (dict(H=(1 << 16) + 1), 2), (dict(T=-1), 1), (dict(T=(1 << 22) + 1), 2), (dict(x=None), 1), (dict(x=P + 1), 1),
    (dict(addend=None), 1), (dict(addend=P + 2), 1), (dict(ws=None), 1), (dict(ws=P + 64), 1), (dict(ws_bytes=512), 1),
])
def test_shared_prefill_refuses(kw, status):
    assert _call(**kw) == status
    assert m.moe_last_error()


def test_shared_prefill_of_no_tokens_is_fine():
    assert _call(T=0, x=None, addend=None, ws=None, ws_bytes=0) == 0


def test_shared_prefill_workspace():
    got = m.moe_shared_prefill_workspace_bytes(4096, 1000, 300)
    assert 300 * (2000 + 4) <= got <= 300 * (2000 + 4) + 512
    assert m.moe_shared_prefill_workspace_bytes(4096, 0, 300) == 0
    assert m.moe_shared_prefill_workspace_bytes(1 << 17, 64, 300) == 0
