"""Products as a prompt's layer uses them, and at the ends of their types: the
shared expert of a prompt, captured and concurrent prompts, the layers of the
4-bit formats, scales and activations at their extremes.  Plain 64-bit forms
and their bounds: product_ref.py."""
import numpy as np
import pytest
import torch

import expert_slot_cache_moe_amd as m
import product_ref as ref
from expert_slot_cache_moe_amd import workloads as W
from expert_slot_cache_moe_amd.layer import SlotCacheLayers

pytestmark = pytest.mark.gpu

FORMATS = [m.MOE_FMT_BF16, m.MOE_FMT_E2M1, m.MOE_FMT_MXFP4]


def _f64(t):
    return t.double().cpu().numpy()


def _bf16(g, shape, scale=1.0):
    return torch.from_numpy(W.normal_bf16(g, shape, scale).view(np.int16)).cuda().view(torch.bfloat16)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _bytes(n):
    return torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- the shared expert of a prompt

@pytest.mark.parametrize("T,H,F", [(1, 64, 32), (7, 45, 17), (100, 130, 70), (300, 1024, 96), (700, 520, 1136),
                                   (2100, 1024, 512)])
def test_shared_prefill_matches_the_plain_form(T, H, F):
    print("shared prefill", T, H, F, flush=True)
    g = W.rng(110, "shared", T, H, F)
    w13, w2, gate = _bf16(g, (2 * F, H), 0.1), _bf16(g, (H, F), 0.1), _bf16(g, (H,), 0.1)
    x = _bf16(g, (T, H))
    add = torch.full((T, H), 77.0, device="cuda")
    sh = m.make_shared(w13.view(-1).view(torch.int16), w2.view(-1).view(torch.int16), gate.view(torch.int16), ffn=F)
    m.moe_shared_prefill(sh, H, x, add, _bytes(m.moe_shared_prefill_workspace_bytes(H, F, T)))
    h, dh = ref.product(_f64(w13), _f64(x), "swiglu")
    dh = dh + (np.abs(h) + dh) * 2.0 ** -8 + 2.0 ** -133              # and its rounding to bf16
    y, a = h @ _f64(w2).T, (np.abs(h) + dh) @ np.abs(_f64(w2)).T
    dy = dh @ np.abs(_f64(w2)).T + F * 2.0 ** -23 * a
    logit, dl = ref.product(_f64(gate)[None], _f64(x))
    s = 1 / (1 + np.exp(-logit))
    # the sigmoid's slope is at most 1/4; exponential, sum and reciprocal: a
    # few roundings each; |logit| 2^-23 of the exponential
    ds = dl / 4 + 2.0 ** -20 * s + s * np.abs(logit) * 2.0 ** -23
    bound = (s + ds) * dy + ds * np.abs(y) + 2.0 ** -23 * np.abs(s * y)
    assert (np.abs(_f64(add) - s * y) <= bound).all()


def test_shared_prefill_is_near_the_shared_expert():
    T, H, F = 40, 1024, 256
    g = W.rng(111, "near")
    sh = m.make_shared(*(torch.from_numpy(W.normal_bf16(g, (n,), 0.05).view(np.int16)).cuda()
                         for n in (2 * F * H, H * F, H)), ffn=F)
    x = _bf16(g, (T, H))
    a, b = torch.zeros((T, H), device="cuda"), torch.zeros((T, H), device="cuda")
    m.moe_shared_prefill(sh, H, x, a, _bytes(m.moe_shared_prefill_workspace_bytes(H, F, T)))
    m.moe_shared_expert(sh, H, x, b, _bytes(m.moe_routed_workspace_bytes(m.MOE_FMT_BF16, H, F, T, 1)))
    # an activation that rounds the other way moves a sum by one of its F terms' 2^-8
    assert np.abs(_f64(a) - _f64(b)).max() <= 2.0 ** -6 * np.abs(_f64(b)).max()


def test_shared_prefill_of_a_nan_row_leaves_the_others():
    T, H, F = 530, 512, 256
    g = W.rng(112, "nan")
    sh = m.make_shared(*(torch.from_numpy(W.normal_bf16(g, (n,), 0.05).view(np.int16)).cuda()
                         for n in (2 * F * H, H * F, H)), ffn=F)
    x = _bf16(g, (T, H))
    outs = []
    for bad in (False, True):
        if bad:
            x[17, 3] = float("nan")
        add = torch.zeros((T, H), device="cuda")
        m.moe_shared_prefill(sh, H, x, add, _bytes(m.moe_shared_prefill_workspace_bytes(H, F, T)))
        outs.append(add)
    keep = torch.arange(T, device="cuda") != 17
    assert torch.isnan(outs[1][17]).all() and torch.equal(outs[0][keep], outs[1][keep])


# ---------------------------------------------------------------- a prompt's layer

class _Prompt:
    """A layer's routed and shared experts over its own buffers."""

    def __init__(self, key, fmt, T, K, P, H, F, Fs):
        g = W.rng(113, *key)
        self.pool = m.make_pool(fmt, H, F, P, W.device_expert_rows(fmt, (113, *key), P, H, F))
        self.sh = m.make_shared(*(torch.from_numpy(W.normal_bf16(g, (n,), 0.05).view(np.int16)).cuda()
                                  for n in (2 * Fs * H, H * Fs, H)), ffn=Fs)
        self.g, self.P, self.H = g, P, H
        self.x, self.w = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, K), device="cuda")
        self.idx = torch.zeros((T, K), dtype=torch.int32, device="cuda")
        self.add = torch.zeros((T, H), device="cuda")
        self.out = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
        self.ws = _bytes(m.moe_routed_prefill_workspace_bytes(fmt, P, H, F, T, K))
        self.ws_shared = _bytes(m.moe_shared_prefill_workspace_bytes(H, Fs, T))
        self.renew()

    def renew(self):
        g, (T, K) = self.g, self.idx.shape
        self.x.copy_(_bf16(g, (T, self.H)))
        self.w.copy_(torch.from_numpy(g.random((T, K)).astype(np.float32)))
        idx = g.integers(0, self.P, (T, K))
        idx[g.random((T, K)) < 0.1] = -1
        self.idx.copy_(_i32(idx))

    def run(self, stream=None):
        m.moe_shared_prefill(self.sh, self.H, self.x, self.add, self.ws_shared, stream=stream)
        m.moe_routed_prefill(self.pool, self.x, self.idx, self.w, self.out, self.ws, addend=self.add, stream=stream)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K", [(1, 4), (600, 6)])
def test_captured_prompt_replays(fmt, T, K):
    p = _Prompt(("replay", fmt, T), fmt, T, K, 20, 256, 128, 96)
    p.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for _ in range(4):
        p.renew()
        p.out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = p.out.clone()
        p.out.fill_(6.0)
        p.run()
        assert torch.equal(got, p.out)


def test_prompts_on_two_streams_at_once():
    ps = [_Prompt(("streams", i), FORMATS[i], 500, 4, 16, 256, 128, 64) for i in range(2)]
    alone = []
    for p in ps:
        p.run()
        torch.cuda.synchronize()
        alone.append(p.out.clone())
        p.out.zero_()
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(ps, streams):
            p.run(stream=s)
    torch.cuda.synchronize()
    for p, e in zip(ps, alone):
        assert torch.equal(p.out, e)


@pytest.mark.parametrize("fmt", FORMATS)
def test_layers_of_each_format_prefill(fmt):
    """SlotCacheLayers.prefill over a pool that the caller holds and over one copied for the call: alike, and
    near the decode step of the same tokens, whose experts are all fetched."""
    L, E, H, F, Fs, T, K = 1, 10, 256, 128, 64, 6, 3
    g = W.rng(114, "layers", fmt)
    rows = [W.expert_rows(fmt, W.rng(114, "rows", fmt, l), E, H, F) for l in range(L)]
    shared = [(W.normal_bf16(g, (2 * Fs * H,), 0.05), W.normal_bf16(g, (H * Fs,), 0.05), W.normal_bf16(g, (H,), 0.05))]
    lay = SlotCacheLayers(layers=L, experts=E, slots=E, hidden=H, ffn=F, fmt=fmt, host_rows=rows, shared=shared,
                          max_tokens=T, max_top_k=K)
    try:
        x = _bf16(g, (T, H))
        logits = torch.from_numpy(g.standard_normal((T, E)).astype(np.float32)).cuda()
        outs = [torch.zeros((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        lay.prefill(0, x, logits, K, outs[0])
        before = m.moe_cache_stats(lay.cache).tolist()
        lay.prefill(0, x, logits, K, outs[1], pool=lay.streamed_pool(0))
        assert m.moe_cache_stats(lay.cache).tolist() == before
        lay.decode(0, x, logits, K, outs[2])
        assert torch.equal(outs[0], outs[1])
        assert np.abs(_f64(outs[0]) - _f64(outs[2])).max() <= 2.0 ** -6 * np.abs(_f64(outs[2])).max()
        for layer in (-1, 1):
            with pytest.raises(ValueError):
                lay.prefill(layer, x, logits, K, outs[0])
        with pytest.raises((ValueError, m.MoeError)):
            lay.prefill(0, x, logits[:4], K, outs[0])
    finally:
        lay.close()


# ---------------------------------------------------------------- the ends of the types

@pytest.mark.parametrize("R", [3, 700])
@pytest.mark.parametrize("scales", [(0, 1, 2), (118, 127, 136), (230, 251, 252), (230, 253, 254)])
def test_mxfp4_scales_at_their_ends(scales, R):
    """Scales from 2^-127 to 2^127, x of a size that keeps the sums in fp32.  Weights from 2^128 on (scales of 2^126
    and 2^127 reach 6 2^127) are past bf16 and fp32 alike: infinities, as moe_dequantize_rows makes them too."""
    n, k = 512, 512
    g = W.rng(115, scales, R)
    codes = g.integers(0, 256, (1, n, k // 2)).astype(np.uint8)
    sc = g.choice(np.array(scales, np.uint8), (1, n, k // 32))
    values = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(n, k)
    w = np.where(nib & 8, -1.0, 1.0) * values[nib & 7] * np.repeat(2.0 ** (sc.astype(float) - 127), 32, -1)[0]
    w[np.abs(w) >= 2.0 ** 128] *= np.inf
    x = _bf16(g, (R, k), 2.0 ** (20 if scales[0] == 0 else 0 if scales[1] == 127 else -40))
    out = torch.zeros((R, n), device="cuda")
    bank = m.make_bank(m.MOE_FMT_MXFP4, torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda())
    m.moe_linear(bank, x, out)
    deq = torch.zeros((n, k), device="cuda")
    m.moe_dequantize_rows(m.MOE_FMT_MXFP4, torch.from_numpy(codes[0]).cuda(), torch.from_numpy(sc[0]).cuda(), deq)
    assert np.array_equal(_f64(deq), w)
    with np.errstate(invalid="ignore"):
        val, bnd = ref.product(w, _f64(x))
    got, fin = _f64(out), np.isfinite(val)
    assert np.isfinite(val).all() == (scales[2] < 253) and np.abs(val[fin]).max(initial=0) < 2.0 ** 127
    assert ref.off(got[fin], val[fin], bnd[fin], "float32") <= 0
    assert np.array_equal(got[~fin], val[~fin], equal_nan=True)


@pytest.mark.parametrize("R", [3, 700])
@pytest.mark.parametrize("small", ["x", "weights"])
def test_bf16_subnormal_operands_count(small, R):
    n, k = 512, 512
    g = W.rng(116, small, R)
    sub = torch.from_numpy(g.integers(-127, 128, (1, n, k) if small == "weights" else (R, k)).astype(np.float32))
    sub = (sub * 2.0 ** -133).to(torch.bfloat16)                 # exact: 7 bits below 2^-126
    sub = sub.cuda()
    other = _bf16(g, (R, k) if small == "weights" else (1, n, k), 2.0 ** 30)
    w, x = (sub, other) if small == "weights" else (other, sub)
    out = torch.zeros((R, n), device="cuda")
    m.moe_linear(m.make_bank(m.MOE_FMT_BF16, w.contiguous()), x, out)
    val, bnd = ref.product(_f64(w)[0], _f64(x))
    assert ref.off(_f64(out), val, bnd, "float32") <= 0


@pytest.mark.parametrize("T", [2, 900])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_at_their_ends(act, T):
    """x is zero, so that each column is the activation of its bias."""
    n, k = 1024, 64
    v = np.array([0.0, -0.0, 1e-38, -1e-38, 1e-20, -1e-20, 0.5, -0.5, 5.0, -5.0, 14.0, -14.0, 87.0, -87.0, 89.0, -89.0,
                  200.0, -200.0, 1e10, -1e10, 3e38, -3e38, np.inf, np.nan], np.float32)
    bias = torch.from_numpy(np.resize(v, (1, n))).cuda()
    g = W.rng(117, act, T)
    bank = m.make_bank(m.MOE_FMT_BF16, _bf16(g, (1, n, k)))
    out = torch.zeros((T, n), device="cuda")
    m.moe_linear(bank, torch.zeros((T, k), dtype=torch.bfloat16, device="cuda"), out, bias=bias.view(-1),
                 activation=m.MOE_ACT_SILU if act == "silu" else m.MOE_ACT_GELU)
    got, y = _f64(out), np.resize(v.astype(np.float64), n)
    assert (got == got[0])[:, ~np.isnan(y)].all()
    with np.errstate(over="ignore", invalid="ignore"):
        val, bnd = ref.activate(y[None], 0 * y[None], act)
    fin = np.isfinite(y)
    assert (np.abs(got[0] - val[0])[fin] <= bnd[0][fin] + np.abs(val[0][fin]) * 2.0 ** -23 + 2.0 ** -126).all()
    assert np.isnan(got[0][np.isnan(y)]).all() and (got[0][y == np.inf] == np.inf).all()


# ---------------------------------------------------------------- short rows of 4 bits

def _decoded(g, fmt, P, n, k):
    """A bank of random codes and finite scales, its parts, and its values."""
    values = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    codes = g.integers(0, 256, (P, n, k // 2)).astype(np.uint8)
    if fmt == m.MOE_FMT_E2M1:
        sc = g.integers(0x28, 0x48, (P, n, k // 16)).astype(np.uint8)
        scale = np.repeat((8 + (sc & 7)) * 2.0 ** ((sc >> 3).astype(float) - 10), 16, -1)
    else:
        sc = g.integers(122, 130, (P, n, k // 32)).astype(np.uint8)
        scale = np.repeat(2.0 ** (sc.astype(float) - 127), 32, -1)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(P, n, k)
    return codes, sc, np.where(nib & 8, -1.0, 1.0) * values[nib & 7] * scale


@pytest.mark.parametrize("fmt", [m.MOE_FMT_E2M1, m.MOE_FMT_MXFP4])
@pytest.mark.parametrize("P,n,k,R", [(1, 4, 32, 17000), (1, 130, 32, 3000), (120, 96, 32, 2400), (2, 67, 64, 5000),
                                     (120, 96, 64, 2400), (3, 257, 96, 3100), (130, 60, 96, 4000), (1, 16, 128, 16000)])
def test_rows_shorter_than_a_span(fmt, P, n, k, R):
    g = W.rng(118, fmt, P, n, k, R)
    codes, sc, w = _decoded(g, fmt, P, n, k)
    bank = m.make_bank(fmt, torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda())
    x = _bf16(g, (R, k))
    offsets = np.concatenate([[0], np.sort(g.integers(0, R + 1, P - 1)), [R]]).astype(np.int32)
    out = torch.full((R, n), 77.0, device="cuda")
    m.moe_grouped_product(bank, x, _i32(offsets), out)
    done, val, bnd = ref.grouped(w, _f64(x), offsets, R)
    assert done.all() and ref.off(_f64(out), val, bnd, "float32") <= 0


@pytest.mark.parametrize("fmt,bad", [(m.MOE_FMT_E2M1, 0x7f), (m.MOE_FMT_MXFP4, 0xff)])
@pytest.mark.parametrize("k", [32, 64, 96])
def test_nan_scales_of_short_rows_stay_in_them(fmt, bad, k):
    P, n, R = 2, 70, 4000
    g = W.rng(119, fmt, k)
    codes, sc, _ = _decoded(g, fmt, P, n, k)
    sc[0, 1] = sc[0, 69] = sc[1, 0] = sc[1, 5] = bad
    bank = m.make_bank(fmt, torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda())
    out = torch.zeros((R, n), device="cuda")
    m.moe_grouped_product(bank, _bf16(g, (R, k)), _i32([0, 2100, R]), out)
    nan = np.zeros((R, n), bool)
    nan[:2100, [1, 69]] = nan[2100:, [0, 5]] = True
    assert np.array_equal(np.isnan(_f64(out)), nan)


# ---------------------------------------------------------------- rows shorter than a vector

@pytest.mark.parametrize("k", [1, 3, 7])
@pytest.mark.parametrize("P,n,R,act", [(300, 40, 600, "none"), (40, 600, 1600, "swiglu"), (60, 300, 6000, "none"),
                                       (1, 2100, 8192, "none"), (1, 2100, 8192, "swiglu"), (1, 3, 9000, "none")])
def test_bf16_rows_shorter_than_a_vector(P, n, k, R, act):
    """A tile reads eight elements at once: here there are fewer, and the buffers end with the last row."""
    print("short rows", P, n, k, R, act, flush=True)
    g = W.rng(120, P, n, k, R, act)
    w, x = _bf16(g, (P, n, k)), _bf16(g, (R, k))
    cols = n // 2 if act == "swiglu" else n
    offsets = np.concatenate([[0], np.sort(g.integers(0, R + 1, P - 1)), [R]]).astype(np.int32)
    out = torch.full((R, cols), 77.0, device="cuda")
    m.moe_grouped_product(m.make_bank(m.MOE_FMT_BF16, w), x, _i32(offsets), out,
                          activation=m.MOE_ACT_SWIGLU if act == "swiglu" else m.MOE_ACT_NONE)
    done, val, bnd = ref.grouped(_f64(w), _f64(x), offsets, R, act=act)
    assert done.all() and ref.off(_f64(out), val, bnd, "float32") <= 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,n,k", [(3, 5, 40), (700, 515, 72), (900, 130, 264), (5000, 1027, 64), (9000, 3, 64)])
def test_odd_rows_of_residuals_in_place(T, n, k, dtype):
    """out as its own residual, rows of an odd number of columns: as with a copy of it, and nothing beside the rows."""
    g = W.rng(121, T, n, k, dtype)
    bank = m.make_bank(m.MOE_FMT_BF16, _bf16(g, (1, n, k)))
    x, res = _bf16(g, (T, k)), _bf16(g, (T, n + 2)).to(dtype)
    out, place = torch.zeros((T, n), dtype=dtype, device="cuda"), res.clone()
    m.moe_linear(bank, x, out, residual=res[:, :n], activation=m.MOE_ACT_SILU)
    m.moe_linear(bank, x, place[:, :n], residual=place[:, :n], activation=m.MOE_ACT_SILU)
    assert torch.equal(place[:, :n], out) and torch.equal(place[:, n:], res[:, n:])
    val, bnd = ref.product(_f64(bank._keep[0])[0], _f64(x), "silu", residual=_f64(res[:, :n]))
    assert ref.off(_f64(out), val, bnd, str(dtype).split(".")[1]) <= 0
