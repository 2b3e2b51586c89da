"""Caller-side buffers for an offloaded MoE stack: pinned host rows per
layer, device slot banks, per-layer shared experts, and the C cache over
them.  Allocation and marshalling only (torch owns the memory); every step
of the layer runs in the HIP library."""
from __future__ import annotations

import numpy as np
import torch

from . import (MOE_FMT_BF16, MOE_FMT_E2M1, MOE_TYPE_BF16, _on_current_device, _rows_of, _type_of, _want, _weights_of,
               make_pool, make_shared, moe_bank_row_bytes, moe_cache_create, moe_cache_destroy, moe_last_error,
               moe_layer_decode, moe_layer_decode_hybrid, moe_layer_decode_router, moe_quantize_rows, moe_route,
               moe_routed_prefill, moe_routed_prefill_workspace_bytes, moe_shared_prefill,
               moe_shared_prefill_workspace_bytes, moe_topk)


def pinned(a: np.ndarray) -> torch.Tensor:
    t = torch.empty(a.shape, dtype=torch.uint8, pin_memory=True)
    t.numpy()[...] = a
    return t


def quantized_banks(fmt, w13, w2, hidden, ffn, device="cuda"):
    """The banks of a 4-bit format, uint8 device tensors [E, row_bytes], for
    experts given in bf16: w13 [E, 2F*H] and w2 [E, H*F] as uint8, int16 or
    bfloat16 rows (numpy or torch).  E2M1 global scales are the matrix's
    largest finite magnitude / (6 * 448), or 1 for a matrix of zeros; a block
    with NaN or infinity is NaN, the others keep their values."""
    banks = []
    for w, n, k in ((w13, 2 * ffn, hidden), (w2, hidden, ffn)):
        t = torch.from_numpy(np.ascontiguousarray(w)) if isinstance(w, np.ndarray) else w
        E = t.shape[0]
        t = t.to(device).contiguous().view(torch.uint8).view(torch.bfloat16).view(E * n, k)
        glob = None
        if fmt == MOE_FMT_E2M1:
            amax = t.abs().nan_to_num_(nan=0.0, posinf=0.0).amax(1).float().view(E, n).amax(1) / (6 * 448)
            glob = torch.where(amax > 0, amax, torch.ones_like(amax))
        blk = 16 if fmt == MOE_FMT_E2M1 else 32
        codes = torch.empty((E * n, k // 2), dtype=torch.uint8, device=device)
        scales = torch.empty((E * n, k // blk), dtype=torch.uint8, device=device)
        moe_quantize_rows(fmt, t, codes, scales, globals=glob, rows_per_global=n if glob is not None else 0)
        banks += [codes.view(E, -1), scales.view(E, -1)]
        if glob is not None:
            banks.append(glob.view(E, 1).view(torch.uint8))
    return banks


class SlotCacheLayers:
    """host_rows[l]: list over banks of uint8 arrays [E, row_bytes] (numpy,
    copied into pinned memory) or pinned uint8 tensors (used as given).
    shared[l]: (w13 [2F*H] u16, w2 [H*F] u16, gate [H] u16) numpy or None.
    router: a moe_router_t for every layer, or a list of them (None: the
    softmax top-k); decode() then routes with it.  quantize: host_rows[l]
    are the two bf16 banks, quantized to the 4-bit fmt here."""

    def __init__(self, *, layers, experts, slots, hidden, ffn, fmt=MOE_FMT_BF16, host_rows,
                 shared=None, max_tokens=1, max_top_k=8, overlap=1, one_call_width=256,
                 query_width=128, max_routes=None, gather_workgroups=0, device="cuda", router=None,
                 quantize=False):
        self.L, self.E, self.S, self.H, self.F, self.fmt = layers, experts, slots, hidden, ffn, fmt
        self.device = torch.device(device)
        self.row_bytes = moe_bank_row_bytes(fmt, hidden, ffn)
        self.host = []
        for l in range(layers):
            banks = []
            rows = host_rows[l]
            if quantize:
                rows = [b.cpu().numpy() for b in quantized_banks(fmt, *rows, hidden, ffn, self.device)]
            for b, a in enumerate(rows):
                t = a if isinstance(a, torch.Tensor) else pinned(np.ascontiguousarray(a))
                assert t.is_pinned() and t.shape == (experts, self.row_bytes[b])
                banks.append(t)
            self.host.append(banks)
        self.slot_banks = [torch.zeros((slots, r), dtype=torch.uint8, device=self.device)
                           for r in self.row_bytes]
        self.shared = None
        if shared is not None:
            self.shared = []
            for l in range(layers):
                if shared[l] is None:
                    self.shared.append(None)
                    continue
                w13, w2, gate = (torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(self.device)
                                 for a in shared[l])
                self.shared.append(make_shared(w13, w2, gate, ffn=w2.numel() // hidden))
        self.routers = list(router) if isinstance(router, (list, tuple)) else [router] * layers
        if len(self.routers) != layers:
            raise ValueError(f"{len(self.routers)} routers for {layers} layers")
        if max_routes is None:
            max_routes = max(max_tokens * max_top_k, 1)
        self.cache = moe_cache_create(
            num_layers=layers, num_experts=experts, num_slots=slots, hidden=hidden, ffn=ffn,
            weight_format=fmt, one_call_width=one_call_width, query_width=query_width,
            max_routes=max_routes, max_tokens=max_tokens, max_top_k=max_top_k, overlap=overlap,
            gather_workgroups=gather_workgroups, host_banks=self.host, slot_banks=self.slot_banks)

    def _shared(self, layer):
        # the library checks the layer; an out-of-range one gets no shared expert here
        if self.shared is None or not 0 <= layer < len(self.shared):
            return None
        return self.shared[layer]

    def decode(self, layer, x, logits, K, out, ids_out=None, w_out=None, max_fetch=-1, stream=None):
        sh = self._shared(layer)
        router = self.routers[layer] if 0 <= layer < len(self.routers) else None
        if router is not None:
            moe_layer_decode_router(self.cache, layer, x, logits, K, out, router=router, shared=sh,
                                    max_fetch=max_fetch, ids_out=ids_out, w_out=w_out, stream=stream)
            return
        moe_layer_decode(self.cache, layer, x, logits, K, out, shared=sh, max_fetch=max_fetch,
                         ids_out=ids_out, w_out=w_out, stream=stream)

    def decode_hybrid(self, layer, x, logits, K, out, ids_out=None, w_out=None, max_fetch=-1,
                      stream=None):
        """decode with the misses on host threads; not with routers, whichever
        layer they are for (a layer without one can be stepped through
        moe_layer_decode_hybrid itself)."""
        if any(r is not None for r in self.routers):
            raise ValueError("the hybrid step routes by softmax top-k; it takes no router")
        sh = self._shared(layer)
        moe_layer_decode_hybrid(self.cache, layer, x, logits, K, out, shared=sh, max_fetch=max_fetch,
                                ids_out=ids_out, w_out=w_out, stream=stream)

    def prefill(self, layer, x, logits, K, out, ids_out=None, w_out=None, pool=None):
        """A prompt's rows through all of the layer's experts, on the current
        stream: the routes of decode(), the shared expert, and
        moe_routed_prefill over `pool` (streamed_pool(layer), copied here if
        not given: the host waits for the copy of all experts, 28 ms for 1.6
        GB, and a capture cannot hold it).  The cache and its statistics
        stay as they are; any number of tokens up to 65535.  x and out are
        bf16 [T, H], logits fp32 [T, E] (rows may be strided if the layer has a
        router), ids_out int32 and w_out fp32 [T, K]; all of that, the sizes
        and the pool's are checked before anything is launched."""
        if not 0 <= layer < self.L:
            raise ValueError(f"layer {layer} outside [0, {self.L})")
        T = x.shape[0]
        _on_current_device(x, logits, out, ids_out, w_out, *_weights_of(self._shared(layer)),
                           *(self.slot_banks if pool is None else _weights_of(pool)))
        router = self.routers[layer]
        for name, t, shape, dtype in (("x", x, (T, self.H), None), ("logits", logits, (T, self.E), torch.float32),
                                      ("out", out, (T, self.H), None), ("ids_out", ids_out, (T, K), torch.int32),
                                      ("w_out", w_out, (T, K), torch.float32)):
            if t is None:
                continue
            if t is logits and router is not None:      # a router takes rows of any stride
                _rows_of(t, name)
                if tuple(t.shape) != shape or t.dtype != dtype:
                    raise ValueError(f"{name}: expected {dtype} of shape {shape}, got {t.dtype} of {tuple(t.shape)}")
                continue
            _want(t, name, shape, dtype)
            if dtype is None and _type_of(t, name) != MOE_TYPE_BF16:
                raise ValueError(f"{name} must be bfloat16")
        if pool is not None and pool.hidden != self.H:
            raise ValueError(f"pool: hidden {pool.hidden}, expected {self.H}")
        n = moe_routed_prefill_workspace_bytes(
            *((self.fmt, self.E, self.H, self.F) if pool is None else
              (pool.weight_format, pool.num_rows, pool.hidden, pool.ffn)), T, K)
        if n == 0:      # sizes that moe_routed_prefill would refuse
            raise ValueError(f"a prompt of {T} tokens, top {K}: {moe_last_error()}")
        ids = torch.empty((T, K), dtype=torch.int32, device=x.device) if ids_out is None else ids_out
        w = torch.empty((T, K), dtype=torch.float32, device=x.device) if w_out is None else w_out
        if router is None:
            moe_topk(logits, K, ids, w)
        else:
            moe_route(router, logits, K, ids, w)
        shared, addend = self._shared(layer), None
        if shared is not None:
            addend = torch.empty((T, self.H), dtype=torch.float32, device=x.device)
            ns = moe_shared_prefill_workspace_bytes(self.H, shared.ffn, T)
            moe_shared_prefill(shared, self.H, x, addend, torch.empty(ns, dtype=torch.uint8, device=x.device))
        if pool is None:
            pool = self.streamed_pool(layer)
        moe_routed_prefill(pool, x, ids, w, out, torch.empty(n, dtype=torch.uint8, device=x.device),
                           addend=addend)

    def streamed_pool(self, layer):
        """The whole layer's experts copied to device memory, rows = expert
        ids: the non-cached reference layer for the routed kernels."""
        banks = [h.to(self.device) for h in self.host[layer]]
        return make_pool(self.fmt, self.H, self.F, self.E, banks)

    def close(self):
        if self.cache is not None:
            moe_cache_destroy(self.cache)
        self.cache = None
        # drop the pinned host store and the slot banks with the cache
        self.host = []
        self.slot_banks = []
        self.shared = None
