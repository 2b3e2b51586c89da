// The C ABI (include/moe_cache.h), part 5: lists of routes by matrix row,
// products grouped by matrix, dense products, and the routed and shared experts
// of a prompt made of them.  Checks on the host, then launches; nothing here
// synchronises or allocates.
#include <algorithm>

#include "moe_api_internal.h"

using namespace moe;
using namespace moe::api;

namespace {

bool known_type(int t) { return t == MOE_TYPE_F32 || t == MOE_TYPE_BF16; }
int type_bytes(int t) { return t == MOE_TYPE_F32 ? 4 : 2; }
bool misaligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

moe_status_t check_lists(int32_t P, int32_t T, int32_t K) {
    if (P < 1 || T < 0 || K < 1) return fail(MOE_INVALID_ARG, "bad lists: %d rows, T=%d K=%d", P, T, K);
    if (P > kListsMaxRows || (int64_t)T * K > kListsMaxRoutes)
        return fail(MOE_UNSUPPORTED, "lists of %lld routes over %d rows", (long long)T * K, P);
    return MOE_OK;
}

// The bank and what a product does to its sums, into p.
moe_status_t check_product(const moe_bank_t *b, int32_t R, int32_t act, int32_t bias_type, const void *bias,
                           int32_t out_type, const void *out, int64_t out_stride, const void *x, int64_t x_stride,
                           ProductParams &p) {
    if (!b) return fail(MOE_INVALID_ARG, "bank is NULL");
    if (b->weight_format != MOE_FMT_BF16 && b->weight_format != MOE_FMT_E2M1 && b->weight_format != MOE_FMT_MXFP4)
        return fail(MOE_INVALID_ARG, "unknown weight format %d", b->weight_format);
    const bool wide = b->weight_format == MOE_FMT_BF16;
    if (b->num_rows < 1 || b->n < 1 || b->k < 1 || (!wide && b->k % 32))
        return fail(MOE_INVALID_ARG, "bad bank: %d matrices of %d x %d%s", b->num_rows, b->n, b->k,
                    wide ? "" : " (4-bit: k a multiple of 32)");
    if (b->num_rows > kProductMaxMatrices || b->n > kProductMaxN || b->k > kProductMaxK)
        return fail(MOE_UNSUPPORTED, "bank of %d matrices of %d x %d", b->num_rows, b->n, b->k);
    if (act != MOE_ACT_NONE && act != MOE_ACT_SILU && act != MOE_ACT_GELU && act != MOE_ACT_SWIGLU)
        return fail(MOE_INVALID_ARG, "unknown activation %d", act);
    if (act == MOE_ACT_SWIGLU && b->n % 2) return fail(MOE_INVALID_ARG, "swiglu needs an even n, got %d", b->n);
    if (!known_type(out_type)) return fail(MOE_INVALID_ARG, "unknown output type %d", out_type);
    if (bias && !known_type(bias_type)) return fail(MOE_INVALID_ARG, "unknown bias type %d", bias_type);
    const int cols = act == MOE_ACT_SWIGLU ? b->n / 2 : b->n;
    if (x_stride < b->k) return fail(MOE_INVALID_ARG, "x stride %lld < k=%d", (long long)x_stride, b->k);
    if (out_stride < cols) return fail(MOE_INVALID_ARG, "out stride %lld < %d", (long long)out_stride, cols);
    if (R < 0) return fail(MOE_INVALID_ARG, "%d rows", R);
    if (R > kProductMaxPlaces) return fail(MOE_UNSUPPORTED, "%d rows > %d", R, kProductMaxPlaces);
    if (!b->weights_dev || misaligned(b->weights_dev, wide ? 2 : 16))
        return fail(MOE_INVALID_ARG, "bank weights are NULL, or not %d-byte aligned", wide ? 2 : 16);
    if (!wide && (!b->scales_dev || misaligned(b->scales_dev, b->weight_format == MOE_FMT_E2M1 ? 2 : 1)))
        return fail(MOE_INVALID_ARG, "bank scales are NULL or misaligned");
    if (misaligned(b->globals_dev, 4)) return fail(MOE_INVALID_ARG, "bank globals are not 4-byte aligned");
    if (b->globals_dev && b->weight_format != MOE_FMT_E2M1)
        return fail(MOE_INVALID_ARG, "only E2M1 banks have global scales");
    if (R > 0 && (!x || !out)) return fail(MOE_INVALID_ARG, "NULL product buffer");
    if (misaligned(x, 2) || misaligned(out, type_bytes(out_type)) || (bias && misaligned(bias, type_bytes(bias_type))))
        return fail(MOE_INVALID_ARG, "product buffers are not aligned to their elements");
    p = ProductParams{};
    p.w = static_cast<const uint8_t *>(b->weights_dev);
    p.scales = static_cast<const uint8_t *>(b->scales_dev);
    p.globals = b->globals_dev;
    p.fmt = b->weight_format;
    p.P = b->num_rows;
    p.n = b->n;
    p.k = b->k;
    p.x = static_cast<const uint16_t *>(x);
    p.x_stride = x_stride;
    p.R = p.x_rows = p.out_rows = R;
    p.G = 1;
    p.gather_div = 1;
    p.act = act;
    p.bias = bias;
    p.bias_type = bias_type;
    p.out = const_cast<void *>(out);
    p.out_type = out_type;
    p.out_stride = out_stride;
    return MOE_OK;
}

// A matrix of a pool's experts as a bank: 0 gate and up, 1 down.
moe_bank_t pool_bank(const moe_pool_t *pool, int which) {
    const int fmt = pool->weight_format, first = which * bank_count(fmt) / 2;
    moe_bank_t b{};
    b.weight_format = fmt;
    b.num_rows = pool->num_rows;
    b.n = which == 0 ? 2 * pool->ffn : pool->hidden;
    b.k = which == 0 ? pool->hidden : pool->ffn;
    b.weights_dev = pool->banks_dev[first];
    if (fmt != MOE_FMT_BF16) b.scales_dev = pool->banks_dev[first + 1];
    if (fmt == MOE_FMT_E2M1) b.globals_dev = static_cast<const float *>(pool->banks_dev[first + 2]);
    return b;
}

moe_status_t check_prefill(int32_t fmt, int32_t P, int32_t H, int32_t F, int32_t T, int32_t K) {
    if (fmt != MOE_FMT_BF16 && fmt != MOE_FMT_E2M1 && fmt != MOE_FMT_MXFP4)
        return fail(MOE_INVALID_ARG, "unknown weight format %d", fmt);
    if (H < 1 || F < 1) return fail(MOE_INVALID_ARG, "hidden %d / ffn %d", H, F);
    if (H > kProductMaxK || F > kProductMaxK || (fmt != MOE_FMT_BF16 && (H % 32 || F % 32)))
        return fail(MOE_UNSUPPORTED, "hidden %d / ffn %d", H, F);
    if (T > 65535) return fail(MOE_UNSUPPORTED, "T=%d > 65535", T);
    if (K > kMaxTopK) return fail(MOE_UNSUPPORTED, "K=%d > %d", K, kMaxTopK);
    return check_lists(P, T, K);
}

// Lists, the activations of every place, the down projections of every route.
struct PrefillWs {
    size_t offsets, order, counts, h, d, total;
};
PrefillWs prefill_ws(int P, int H, int F, int T, int K) {
    const size_t n = (size_t)T * K;
    PrefillWs w;
    w.offsets = 0;
    w.order = w.offsets + align_up(((size_t)P + 1) * 4);
    w.counts = w.order + align_up(n * 4);
    w.h = w.counts + align_up(lists_workspace_bytes(P, (int64_t)n));
    w.d = w.h + align_up(n * F * 2);
    w.total = w.d + align_up(n * H * 4);
    return w;
}

// The activations of every token, and what its gate says.
struct SharedWs {
    size_t h, gate, total;
};
SharedWs shared_ws(int F, int T) {
    SharedWs w;
    w.h = 0;
    w.gate = align_up((size_t)T * F * 2);
    w.total = w.gate + align_up((size_t)T * 4);
    return w;
}

moe_status_t check_shared_prefill(int32_t H, int32_t F, int32_t T) {
    if (H < 1 || F < 1 || T < 0) return fail(MOE_INVALID_ARG, "shared expert: hidden %d / ffn %d, T=%d", H, F, T);
    if (H > kProductMaxK || F > kProductMaxK || T > kProductMaxPlaces)
        return fail(MOE_UNSUPPORTED, "shared expert: hidden %d / ffn %d, T=%d", H, F, T);
    return MOE_OK;
}

}  // namespace

extern "C" {

int64_t moe_group_routes_workspace_bytes(int32_t P, int32_t T, int32_t K) {
    if (check_lists(P, T, K) != MOE_OK) return 0;
    return (int64_t)lists_workspace_bytes(P, (int64_t)T * K);
}

moe_status_t moe_group_routes(const int32_t *idx, int32_t T, int32_t K, int32_t P, int32_t *offsets, int32_t *order,
                              void *ws, int64_t ws_bytes, void *stream) {
    moe_status_t st = check_lists(P, T, K);
    if (st != MOE_OK) return st;
    if (!offsets || (T > 0 && (!idx || !order))) return fail(MOE_INVALID_ARG, "NULL lists buffer");
    const size_t need = lists_workspace_bytes(P, (int64_t)T * K);
    if (ws_bytes < (int64_t)need || (need > 0 && !ws))
        return fail(MOE_INVALID_ARG, "workspace %lld B < %zu B", (long long)ws_bytes, need);
    if (misaligned(idx, 4) || misaligned(offsets, 4) || misaligned(order, 4) || (need > 0 && misaligned(ws, 4)))
        return fail(MOE_INVALID_ARG, "lists buffers are not 4-byte aligned");
    HIP_TRY(launch_lists(idx, T * K, P, offsets, order, static_cast<int32_t *>(ws), static_cast<hipStream_t>(stream)),
            "route lists launch");
    return MOE_OK;
}

moe_status_t moe_grouped_product(const moe_bank_t *bank, const void *x, int64_t x_stride, int32_t x_rows,
                                 const int32_t *offsets, int32_t G, const int32_t *matrices, const int32_t *gather,
                                 int32_t gather_div, const int32_t *scatter, int32_t R, int32_t act,
                                 int32_t bias_type, const void *bias, int32_t out_type, void *out,
                                 int64_t out_stride, int32_t out_rows, void *stream) {
    ProductParams p;
    moe_status_t st = check_product(bank, R, act, bias_type, bias, out_type, out, out_stride, x, x_stride, p);
    if (st != MOE_OK) return st;
    if (G < 1) return fail(MOE_INVALID_ARG, "%d groups", G);
    if (G > kProductMaxMatrices) return fail(MOE_UNSUPPORTED, "%d groups > %d", G, kProductMaxMatrices);
    if (!offsets) return fail(MOE_INVALID_ARG, "offsets is NULL");
    if (!matrices && G > p.P) return fail(MOE_INVALID_ARG, "%d groups over %d matrices without their ids", G, p.P);
    if (gather_div < 1) return fail(MOE_INVALID_ARG, "gather_div %d", gather_div);
    if (x_rows < (gather ? (R > 0) : R)) return fail(MOE_INVALID_ARG, "%d rows of x for %d places", x_rows, R);
    if (out_rows < (scatter ? 0 : R)) return fail(MOE_INVALID_ARG, "%d rows of out for %d places", out_rows, R);
    if (misaligned(offsets, 4) || misaligned(matrices, 4) || misaligned(gather, 4) || misaligned(scatter, 4))
        return fail(MOE_INVALID_ARG, "index buffers are not 4-byte aligned");
    if (R == 0) return MOE_OK;
    p.x_rows = x_rows;
    p.offsets = offsets;
    p.G = G;
    p.matrices = matrices;
    p.gather = gather;
    p.gather_div = gather ? gather_div : 1;
    p.scatter = scatter;
    p.out_rows = out_rows;
    if (!product_launchable(p)) return fail(MOE_UNSUPPORTED, "%d rows of %d x %d: too many tiles", R, p.n, p.k);
    HIP_TRY(launch_product(p, static_cast<hipStream_t>(stream)), "grouped product launch");
    return MOE_OK;
}

moe_status_t moe_linear(const moe_bank_t *bank, const void *x, int64_t x_stride, int32_t T, int32_t act,
                        int32_t bias_type, const void *bias, int32_t res_type, const void *residual,
                        int64_t res_stride, int32_t out_type, void *out, int64_t out_stride, void *stream) {
    ProductParams p;
    moe_status_t st = check_product(bank, T, act, bias_type, bias, out_type, out, out_stride, x, x_stride, p);
    if (st != MOE_OK) return st;
    if (p.P != 1) return fail(MOE_INVALID_ARG, "a dense product takes a bank of one matrix, got %d", p.P);
    if (residual) {
        if (!known_type(res_type)) return fail(MOE_INVALID_ARG, "unknown residual type %d", res_type);
        const int cols = act == MOE_ACT_SWIGLU ? p.n / 2 : p.n;
        if (res_stride < cols) return fail(MOE_INVALID_ARG, "residual stride %lld < %d", (long long)res_stride, cols);
        if (misaligned(residual, type_bytes(res_type)))
            return fail(MOE_INVALID_ARG, "residual is not aligned to its elements");
        p.residual = residual;
        p.res_type = res_type;
        p.res_stride = res_stride;
    }
    if (T == 0) return MOE_OK;
    if (!product_launchable(p)) return fail(MOE_UNSUPPORTED, "%d rows of %d x %d: too many tiles", T, p.n, p.k);
    HIP_TRY(launch_product(p, static_cast<hipStream_t>(stream)), "dense product launch");
    return MOE_OK;
}

int64_t moe_routed_prefill_workspace_bytes(int32_t fmt, int32_t P, int32_t H, int32_t F, int32_t T, int32_t K) {
    if (check_prefill(fmt, P, H, F, T, K) != MOE_OK) return 0;
    return (int64_t)prefill_ws(P, H, F, T, K).total;
}

moe_status_t moe_routed_prefill(const moe_pool_t *pool, const void *x, const int32_t *idx, const float *w, int32_t T,
                                int32_t K, const float *addend, void *out, void *ws, int64_t ws_bytes, void *stream) {
    if (!pool) return fail(MOE_INVALID_ARG, "pool is NULL");
    const int P = pool->num_rows, H = pool->hidden, F = pool->ffn;
    moe_status_t st = check_prefill(pool->weight_format, P, H, F, T, K);
    if (st != MOE_OK) return st;
    for (int b = 0; b < bank_count(pool->weight_format); ++b)
        if (!pool->banks_dev[b]) return fail(MOE_INVALID_ARG, "pool bank %d is NULL", b);
    if (T > 0 && (!x || !idx || !w || !out || !ws)) return fail(MOE_INVALID_ARG, "NULL routed buffer");
    if (misaligned(idx, 4) || misaligned(w, 4) || misaligned(addend, 4) || misaligned(out, 2))
        return fail(MOE_INVALID_ARG, "routed buffers are not aligned to their elements");
    if (misaligned(ws, 256)) return fail(MOE_INVALID_ARG, "workspace must be 256-byte aligned");
    const PrefillWs L = prefill_ws(P, H, F, T, K);
    if (ws_bytes < (int64_t)L.total)
        return fail(MOE_INVALID_ARG, "workspace %lld B < %zu B", (long long)ws_bytes, L.total);
    const moe_bank_t up_bank = pool_bank(pool, 0), down_bank = pool_bank(pool, 1);
    uint8_t *base = static_cast<uint8_t *>(ws);
    uint16_t *h = reinterpret_cast<uint16_t *>(base + L.h);
    float *d = reinterpret_cast<float *>(base + L.d);
    int32_t *offsets = reinterpret_cast<int32_t *>(base + L.offsets), *order = reinterpret_cast<int32_t *>(base + L.order);
    const int R = T * K;
    ProductParams up, down;
    st = check_product(&up_bank, R, MOE_ACT_SWIGLU, 0, nullptr, MOE_TYPE_BF16, h, F, x, H, up);
    if (st == MOE_OK)
        st = check_product(&down_bank, R, MOE_ACT_NONE, 0, nullptr, MOE_TYPE_F32, d, H, h, F, down);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    up.x_rows = T;
    up.gather = order;
    up.gather_div = K;
    down.scatter = order;
    for (ProductParams *p : {&up, &down}) {
        p->offsets = offsets;
        p->G = P;
        if (!product_launchable(*p))
            return fail(MOE_UNSUPPORTED, "%d routes of hidden %d, ffn %d: too many tiles", R, H, F);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    HIP_TRY(launch_lists(idx, R, P, offsets, order, reinterpret_cast<int32_t *>(base + L.counts), s),
            "route lists launch");
    HIP_TRY(launch_product(up, s), "gate/up product launch");
    HIP_TRY(launch_product(down, s), "down product launch");
    HIP_TRY(launch_combine(idx, w, T, K, H, P, d, addend, static_cast<uint16_t *>(out), s), "combine launch");
    return MOE_OK;
}

int64_t moe_shared_prefill_workspace_bytes(int32_t H, int32_t F, int32_t T) {
    if (check_shared_prefill(H, F, T) != MOE_OK) return 0;
    return (int64_t)shared_ws(F, T).total;
}

moe_status_t moe_shared_prefill(const moe_shared_t *sh, int32_t H, const void *x, int32_t T, float *addend, void *ws,
                                int64_t ws_bytes, void *stream) {
    if (!sh) return fail(MOE_INVALID_ARG, "shared expert is NULL");
    const int F = sh->ffn;
    moe_status_t st = check_shared_prefill(H, F, T);
    if (st != MOE_OK) return st;
    if (!sh->w13_dev || !sh->w2_dev || !sh->gate_dev)
        return fail(MOE_INVALID_ARG, "shared expert has a NULL weight");
    if (T > 0 && (!x || !addend || !ws)) return fail(MOE_INVALID_ARG, "NULL shared buffer");
    if (misaligned(ws, 256)) return fail(MOE_INVALID_ARG, "workspace must be 256-byte aligned");
    const SharedWs L = shared_ws(F, T);
    if (ws_bytes < (int64_t)L.total)
        return fail(MOE_INVALID_ARG, "workspace %lld B < %zu B", (long long)ws_bytes, L.total);
    uint16_t *h = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(ws) + L.h);
    float *logits = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + L.gate);
    auto bank = [](const void *w, int n, int k) {
        moe_bank_t b{};
        b.weight_format = MOE_FMT_BF16;
        b.num_rows = 1;
        b.n = n;
        b.k = k;
        b.weights_dev = w;
        return b;
    };
    const moe_bank_t gate_bank = bank(sh->gate_dev, 1, H), up_bank = bank(sh->w13_dev, 2 * F, H),
                     down_bank = bank(sh->w2_dev, H, F);
    ProductParams gate, up, down;
    st = check_product(&gate_bank, T, MOE_ACT_NONE, 0, nullptr, MOE_TYPE_F32, logits, 1, x, H, gate);
    if (st == MOE_OK) st = check_product(&up_bank, T, MOE_ACT_SWIGLU, 0, nullptr, MOE_TYPE_BF16, h, F, x, H, up);
    if (st == MOE_OK) st = check_product(&down_bank, T, MOE_ACT_NONE, 0, nullptr, MOE_TYPE_F32, addend, H, h, F, down);
    if (st != MOE_OK || T == 0) return st;
    down.gate = logits;
    for (const ProductParams *p : {&gate, &up, &down})
        if (!product_launchable(*p))
            return fail(MOE_UNSUPPORTED, "%d tokens of hidden %d, ffn %d: too many tiles", T, H, F);
    hipStream_t s = static_cast<hipStream_t>(stream);
    HIP_TRY(launch_product(gate, s), "shared gate launch");
    HIP_TRY(launch_product(up, s), "shared gate/up product launch");
    HIP_TRY(launch_product(down, s), "shared down product launch");
    return MOE_OK;
}

}  // extern "C"
