"""What SlotCacheLayers.prefill takes and refuses: logits cut out of a wider
buffer, no tokens, and calls that must leave their outputs as they were."""
import numpy as np
import pytest
import torch

import expert_slot_cache_moe_amd as m
from expert_slot_cache_moe_amd import workloads as W
from expert_slot_cache_moe_amd.layer import SlotCacheLayers

pytestmark = pytest.mark.gpu

L, E, H, F, K = 2, 12, 128, 64, 3


def _bf16(g, shape, scale=1.0):
    return torch.from_numpy(W.normal_bf16(g, shape, scale).view(np.int16)).cuda().view(torch.bfloat16)


@pytest.fixture(scope="module")
def layers():
    """Two layers, the second with a router; a shared expert in the first."""
    g = W.rng(150, "layers")
    rows = [W.expert_rows(m.MOE_FMT_BF16, W.rng(150, "rows", l), E, H, F) for l in range(L)]
    shared = [(W.normal_bf16(g, (2 * F * H,), 0.05), W.normal_bf16(g, (H * F,), 0.05), W.normal_bf16(g, (H,), 0.05)),
              None]
    lay = SlotCacheLayers(layers=L, experts=E, slots=4, hidden=H, ffn=F, host_rows=rows, shared=shared, max_tokens=8,
                          max_top_k=K, router=[None, m.make_router(score=m.MOE_SCORE_SIGMOID)])
    yield lay
    lay.close()


def _inputs(T, key):
    g = W.rng(151, T, key)
    return _bf16(g, (T, H)), torch.from_numpy(g.standard_normal((T, E)).astype(np.float32)).cuda()


@pytest.mark.parametrize("T", [2, 7, 90])
def test_logits_cut_out_of_a_wider_buffer(layers, T):
    """A router takes rows of any stride; the plain top-k refuses them."""
    x, logits = _inputs(T, "padded")
    wide = torch.full((T, E + 5), 50.0, device="cuda")        # past the row: the largest there are
    wide[:, :E] = logits
    outs = []
    for lg in (logits, wide[:, :E]):
        out = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
        ids = torch.zeros((T, K), dtype=torch.int32, device="cuda")
        w = torch.zeros((T, K), device="cuda")
        layers.prefill(1, x, lg, K, out, ids_out=ids, w_out=w)
        outs.append((ids, w, out))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        layers.prefill(0, x, wide[:, :E], K, outs[0][2])


@pytest.mark.parametrize("layer", range(L))
def test_no_tokens(layers, layer):
    x, logits = _inputs(1, "none")
    layers.prefill(layer, x[:0], logits[:0], K, torch.zeros((0, H), dtype=torch.bfloat16, device="cuda"))


def test_a_pool_of_another_format_and_width(layers):
    """The pool's own sizes count: experts twice as wide, in MXFP4, under a layer of bf16 ones."""
    T, wide = 40, 2 * F
    pool = m.make_pool(m.MOE_FMT_MXFP4, H, wide, E, W.device_expert_rows(m.MOE_FMT_MXFP4, (152, "wide"), E, H, wide))
    x, logits = _inputs(T, "wide")
    out, e = (torch.zeros((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids, w = torch.zeros((T, K), dtype=torch.int32, device="cuda"), torch.zeros((T, K), device="cuda")
    layers.prefill(1, x, logits, K, out, ids_out=ids, w_out=w, pool=pool)
    n = m.moe_routed_prefill_workspace_bytes(m.MOE_FMT_MXFP4, E, H, wide, T, K)
    m.moe_routed_prefill(pool, x, ids, w, e, torch.empty(n, dtype=torch.uint8, device="cuda"))
    assert torch.equal(out, e) and out.any()


@pytest.mark.parametrize("layer", range(L))
def test_refused_calls_leave_their_outputs(layers, layer):
    T = 9
    x, logits = _inputs(T, "refused")
    out = torch.full((T, H), 77.0, dtype=torch.bfloat16, device="cuda")
    wide_ids = torch.full((T, K + 2), -7, dtype=torch.int32, device="cuda")
    wide_w = torch.full((T, K + 2), -7.0, device="cuda")
    ids, w = wide_ids.view(-1)[:T * K].view(T, K), wide_w.view(-1)[:T * K].view(T, K)
    many = 65536
    xs, ls = _inputs(many, "many")
    ids_many = torch.full((many, K), -7, dtype=torch.int32, device="cuda")
    other = m.make_pool(m.MOE_FMT_BF16, 2 * H, F, E, layers.streamed_pool(layer)._keep)     # (never followed)
    bad = [
        dict(x=x.float()), dict(out=out.float()), dict(x=torch.cat([x, x], 1)[:, :H]),
        dict(out=torch.cat([out, out], 1)[:, :H]), dict(ids_out=wide_ids[:, :K]), dict(w_out=wide_w[:, :K]),
        dict(ids_out=ids.long()), dict(logits=logits.to(torch.bfloat16)), dict(logits=logits.t().contiguous().t()),
        dict(x=x.cpu()), dict(K=E + 1), dict(K=0), dict(pool=other), dict(x=x[:4]),
        dict(x=xs, logits=ls, out=torch.full((many, H), 77.0, dtype=torch.bfloat16, device="cuda"), ids_out=ids_many,
             w_out=None),
    ]
    for kw in bad:
        a = dict(x=x, logits=logits, K=K, out=out, ids_out=ids, w_out=w)
        a.update(kw)
        with pytest.raises((ValueError, m.MoeError)):
            layers.prefill(layer, **a)
            pytest.fail(f"taken: {list(kw)}")
        torch.cuda.synchronize()
        assert (out == 77).all() and (a["out"] == 77).all(), list(kw)
        assert (wide_ids == -7).all() and (wide_w == -7).all() and (ids_many == -7).all(), list(kw)
