"""What the binding of the products and the lists checks by itself.  No GPU:
tensors in host memory stand for the device's, and calls that would launch
have no rows."""
import pytest
import torch

import expert_slot_cache_moe_amd as m

P = 1 << 20      # stands for a device pointer; never followed


@pytest.fixture
def checked(monkeypatch):
    """The tensors whose device was checked."""
    seen = []

    def on_current_device(*tensors):
        m._load_torch()
        seen.extend(t for t in tensors if t is not None)
        return -1                                   # what get_device() says of host memory

    monkeypatch.setattr(m, "_on_current_device", on_current_device)
    monkeypatch.setattr(m, "_stream_on", lambda dev, stream: None)
    monkeypatch.setattr(m, "_dev_ptr", lambda t: None if t is None else P)
    return seen


def _by_hand(num_rows=1, n=32, k=64):
    """A bank whose fields a program has filled itself, as C's callers do."""
    b = m.moe_bank_t()
    b.weight_format, b.num_rows, b.n, b.k, b.weights_dev = m.MOE_FMT_BF16, num_rows, n, k, P
    return b


def test_a_bank_filled_by_hand_is_taken(checked):
    x, out = torch.zeros((0, 64), dtype=torch.bfloat16), torch.zeros((0, 32))
    m.moe_linear(_by_hand(), x, out)
    m.moe_grouped_product(_by_hand(4), x, torch.zeros(5, dtype=torch.int32), out)


def test_a_banks_tensors_are_checked_where_it_has_them(checked):
    w = torch.zeros((1, 32, 64), dtype=torch.bfloat16)
    bank = m.make_bank(m.MOE_FMT_BF16, w)
    checked.clear()
    bank._device = 1                                # made on another device
    m.moe_linear(bank, torch.zeros((0, 64), dtype=torch.bfloat16), torch.zeros((0, 32)))
    assert any(t is w for t in checked)


def _pool(banks):
    return m.make_pool(m.MOE_FMT_BF16, 64, 32, 4, banks)


def test_the_device_of_a_prompts_weights_is_checked(checked):
    """moe_routed_prefill's pool, moe_shared_prefill's matrices; addresses and what is filled by hand say nothing."""
    x, out = torch.zeros((0, 64), dtype=torch.bfloat16), torch.zeros((0, 64), dtype=torch.bfloat16)
    idx, w = torch.zeros((0, 2), dtype=torch.int32), torch.zeros((0, 2))
    ws = torch.zeros(m.moe_routed_prefill_workspace_bytes(m.MOE_FMT_BF16, 4, 64, 32, 0, 2), dtype=torch.uint8)
    banks = [torch.zeros((4, 8), dtype=torch.uint8) for _ in range(2)]
    m.moe_routed_prefill(_pool(banks), x, idx, w, out, ws)
    assert all(any(t is b for t in checked) for b in banks)
    m.moe_routed_prefill(_pool([P, banks[1]]), x, idx, w, out, ws)
    by_hand = m.moe_pool_t()
    by_hand.weight_format, by_hand.hidden, by_hand.ffn, by_hand.num_rows = m.MOE_FMT_BF16, 64, 32, 4
    by_hand.banks_dev[0] = by_hand.banks_dev[1] = P
    m.moe_routed_prefill(by_hand, x, idx, w, out, ws)
    checked.clear()
    parts = [torch.zeros(8, dtype=torch.int16) for _ in range(3)]
    m.moe_shared_prefill(m.make_shared(*parts, ffn=32), 64, x, torch.zeros((0, 64)), ws)
    assert all(any(t is b for t in checked) for b in parts)


MANY = (1 << 32) + 5          # 5 to a call that takes 32 bits


def _many(cols, dtype=torch.bfloat16):
    """A tensor of 2^32 + 5 rows without memory."""
    return torch.empty((MANY, cols), dtype=dtype, device="meta")


def test_more_rows_than_a_call_can_count_are_refused(checked):
    """Counts go to the library in 32 bits: a longer one is refused, not cut to its low bits."""
    i32 = torch.int32
    x, out, off = torch.zeros((8, 64), dtype=torch.bfloat16), torch.zeros((8, 32)), torch.zeros(2, dtype=i32)
    bank = _by_hand()
    idx = torch.zeros((8, 2), dtype=i32)
    refused = [
        lambda: m.moe_linear(bank, _many(64), _many(32)),
        lambda: m.moe_grouped_product(bank, _many(64), off, out, gather=torch.zeros(8, dtype=i32)),
        lambda: m.moe_grouped_product(bank, x, off, _many(32), scatter=torch.zeros(8, dtype=i32)),
        lambda: m.moe_grouped_product(bank, x, off, out, gather=_many(1, i32).view(-1)),
        lambda: m.moe_grouped_product(bank, x, off, out, scatter=_many(1, i32).view(-1)),
        lambda: m.moe_grouped_product(bank, x, _many(1, i32).view(-1), out, matrices=_many(1, i32).view(-1)[:-1]),
        lambda: m.moe_grouped_product(bank, x, off, out, gather=torch.zeros(8, dtype=i32), gather_div=(1 << 32) + 1),
        lambda: m.moe_group_routes(_many(1, i32), 4, torch.zeros(5, dtype=i32), _many(1, i32).view(-1)),
        lambda: m.moe_routed_prefill(_pool([]), _many(64), _many(2, i32), _many(2, torch.float32), _many(64), x),
        lambda: m.moe_shared_prefill(m.make_shared(None, None, None, ffn=32), 64, _many(64), _many(64, torch.float32), x),
        lambda: m.make_bank(m.MOE_FMT_BF16, torch.empty((1, MANY, 2), dtype=torch.bfloat16, device="meta")),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError, match="31 bits"):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises((ValueError, m.MoeError)):
        m.moe_group_routes(idx, (1 << 32) + 4, torch.zeros(5, dtype=i32), torch.zeros(16, dtype=i32))
