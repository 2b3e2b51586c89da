// The C ABI (include/moe_cache.h), part 4: scored routing, 4-bit rows, and
// the MXFP4 products over pool rows.  Checks on the host, then launches;
// nothing here synchronises or allocates.
#include <algorithm>
#include <cmath>

#include "moe_api_internal.h"

using namespace moe;
using namespace moe::api;

namespace moe {
namespace api {

moe_status_t check_router(const moe_router_t *r, int32_t E, RouteParams &p) {
    if (!r) return fail(MOE_INVALID_ARG, "router is NULL");
    if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID)
        return fail(MOE_INVALID_ARG, "unknown score %d", r->score);
    if (r->group_score != MOE_GROUP_MAX && r->group_score != MOE_GROUP_TOP2)
        return fail(MOE_INVALID_ARG, "unknown group score %d", r->group_score);
    if (r->renormalize != 0 && r->renormalize != 1) return fail(MOE_INVALID_ARG, "renormalize must be 0 or 1");
    if (!std::isfinite(r->scale)) return fail(MOE_INVALID_ARG, "the router's scale is not finite");
    if (r->num_groups < 1 || E % r->num_groups)
        return fail(MOE_INVALID_ARG, "%d groups do not divide %d experts", r->num_groups, E);
    if (r->top_groups < 1 || r->top_groups > r->num_groups)
        return fail(MOE_INVALID_ARG, "top_groups %d outside [1, %d]", r->top_groups, r->num_groups);
    if (reinterpret_cast<uintptr_t>(r->bias_dev) % 4) return fail(MOE_INVALID_ARG, "bias is not 4-byte aligned");
    if (E > kRouteMaxExperts) return fail(MOE_UNSUPPORTED, "%d experts > %d", E, kRouteMaxExperts);
    if (r->num_groups > kRouteMaxGroups)
        return fail(MOE_UNSUPPORTED, "%d groups > %d", r->num_groups, kRouteMaxGroups);
    p = RouteParams{};
    p.score = r->score;
    // every group kept: the groups decide nothing
    p.num_groups = r->top_groups == r->num_groups ? 1 : r->num_groups;
    p.top_groups = p.num_groups == 1 ? 1 : r->top_groups;
    p.group_score = r->group_score;
    p.renormalize = r->renormalize;
    p.scale = r->scale;
    p.bias = r->bias_dev;
    while ((1 << p.log_groups) < p.num_groups) ++p.log_groups;
    const uint64_t gs = (uint64_t)(E / p.num_groups);
    p.group_magic = gs > 1 ? (uint32_t)(((1ull << 32) + gs - 1) / gs) : 0u;
    return MOE_OK;
}

}  // namespace api
}  // namespace moe

namespace {

bool known_type(int t) { return t == MOE_TYPE_F32 || t == MOE_TYPE_BF16; }
int type_bytes(int t) { return t == MOE_TYPE_F32 ? 4 : 2; }

// The checks quantise and dequantise share; `dense` is the float side.
moe_status_t check_rows(int32_t fmt, int32_t type, const void *dense, int64_t stride, int64_t rows, int32_t cols,
                        const float *globals, int64_t per, const void *codes, const void *scales, RowsParams &p) {
    if (fmt != MOE_FMT_MXFP4 && fmt != MOE_FMT_E2M1)
        return fail(MOE_INVALID_ARG, "weight format %d is not a 4-bit format", fmt);
    if (!known_type(type)) return fail(MOE_INVALID_ARG, "unknown element type %d", type);
    const int blk = fmt == MOE_FMT_MXFP4 ? 32 : 16;
    if (rows < 0 || cols < 1 || cols % blk)
        return fail(MOE_INVALID_ARG, "bad rows %lld x cols %d (cols: multiples of %d)", (long long)rows, cols, blk);
    // the kernels' divisions by multiplication hold for products below 2^64
    if (rows > ((int64_t)1 << 32) || cols > (1 << 19))
        return fail(MOE_UNSUPPORTED, "%lld rows of %d", (long long)rows, cols);
    if (stride < cols) return fail(MOE_INVALID_ARG, "row stride %lld < cols %d", (long long)stride, cols);
    if (globals && fmt != MOE_FMT_E2M1) return fail(MOE_INVALID_ARG, "only E2M1 rows have global scales");
    if (globals && per < 1) return fail(MOE_INVALID_ARG, "rows_per_global %lld", (long long)per);
    if (rows > 0) {
        if (!dense || !codes || !scales) return fail(MOE_INVALID_ARG, "NULL rows buffer");
        if (reinterpret_cast<uintptr_t>(dense) % type_bytes(type))
            return fail(MOE_INVALID_ARG, "dense rows are not aligned to their elements");
        if (reinterpret_cast<uintptr_t>(codes) % (blk / 2))
            return fail(MOE_INVALID_ARG, "codes must be %d-byte aligned", blk / 2);
        if (reinterpret_cast<uintptr_t>(globals) % 4) return fail(MOE_INVALID_ARG, "globals are not 4-byte aligned");
    }
    p = RowsParams{};
    p.rows = rows;
    p.cols = cols;
    p.stride = stride;
    p.globals = globals;
    p.rows_per_global = globals ? std::min<int64_t>(per, (int64_t)1 << 32) : 1;
    return MOE_OK;
}

// Sizes of a product, pointers aside.
moe_status_t check_mx_sizes(int32_t P, int32_t n, int32_t k, int32_t T, int32_t K) {
    if (P < 1 || n < 1 || k < 32 || k % 32)
        return fail(MOE_INVALID_ARG, "bad MXFP4 bank: %d matrices of %d x %d", P, n, k);
    if (T < 0 || K < 1) return fail(MOE_INVALID_ARG, "bad T=%d K=%d", T, K);
    if (P > kMxMaxRows || n > kMxMaxN || k > kMxMaxK)
        return fail(MOE_UNSUPPORTED, "MXFP4 bank of %d matrices of %d x %d", P, n, k);
    if (K > kMaxTopK) return fail(MOE_UNSUPPORTED, "K=%d > %d", K, kMaxTopK);
    if ((int64_t)T * K > kMxMaxRoutes)
        return fail(MOE_UNSUPPORTED, "T*K=%lld > %d routes", (long long)T * K, kMxMaxRoutes);
    return MOE_OK;
}

moe_status_t check_routed_mx_sizes(int32_t P, int32_t H, int32_t F, int32_t T, int32_t K) {
    if (H < 1 || F < 1) return fail(MOE_INVALID_ARG, "hidden %d / ffn %d", H, F);
    if (F > kMxMaxN / 2) return fail(MOE_UNSUPPORTED, "ffn %d > %d", F, kMxMaxN / 2);
    if (H % 32 || F % 32) return fail(MOE_UNSUPPORTED, "hidden %d / ffn %d are not multiples of 32", H, F);
    if (T > 65535) return fail(MOE_UNSUPPORTED, "T=%d > 65535", T);
    moe_status_t st = check_mx_sizes(P, 2 * F, H, T, K);
    return st != MOE_OK ? st : check_mx_sizes(P, H, F, T * K, 1);
}

// The products' workspace (one region, used by the two in turn), the
// activations of every route, and their down projections.
struct RoutedMxWs {
    size_t h, d, total;
};
RoutedMxWs routed_mx_ws(int P, int H, int F, int T, int K) {
    const size_t n = (size_t)T * K;
    RoutedMxWs w;
    w.h = std::max(mx_workspace_bytes(P, 2 * F, H, T, K), mx_workspace_bytes(P, H, F, T * K, 1));
    w.d = w.h + align_up(n * F * 2);
    w.total = w.d + align_up(n * H * 4);
    return w;
}

}  // namespace

extern "C" {

moe_status_t moe_route(const moe_router_t *router, int32_t logits_type, const void *logits, int64_t stride,
                       int32_t T, int32_t E, int32_t K, int32_t *ids, float *w, void *stream) {
    if (!known_type(logits_type)) return fail(MOE_INVALID_ARG, "unknown logits type %d", logits_type);
    if (T < 0 || E < 1 || K < 1 || K > E || K > kMaxTopK)
        return fail(MOE_INVALID_ARG, "bad routing sizes T=%d E=%d K=%d", T, E, K);
    if (stride < E) return fail(MOE_INVALID_ARG, "row stride %lld < E=%d", (long long)stride, E);
    if (T > kRouteMaxRows) return fail(MOE_UNSUPPORTED, "T=%d > %d", T, kRouteMaxRows);
    RouteParams p;
    moe_status_t st = check_router(router, E, p);
    if (st != MOE_OK) return st;
    if (T > 0 && (!logits || !ids || !w)) return fail(MOE_INVALID_ARG, "NULL routing buffer");
    if (reinterpret_cast<uintptr_t>(logits) % type_bytes(logits_type) || reinterpret_cast<uintptr_t>(ids) % 4 ||
        reinterpret_cast<uintptr_t>(w) % 4)
        return fail(MOE_INVALID_ARG, "routing buffers are not aligned to their elements");
    HIP_TRY(launch_route(p, logits_type, logits, stride, T, E, K, ids, w, static_cast<hipStream_t>(stream)),
            "route launch");
    return MOE_OK;
}

moe_status_t moe_quantize_rows(int32_t fmt, int32_t type, const void *src, int64_t stride, int64_t rows,
                               int32_t cols, const float *globals, int64_t per, void *codes, void *scales,
                               void *stream) {
    RowsParams p;
    moe_status_t st = check_rows(fmt, type, src, stride, rows, cols, globals, per, codes, scales, p);
    if (st != MOE_OK) return st;
    HIP_TRY(launch_quantize(fmt, type, p, src, static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales),
                            static_cast<hipStream_t>(stream)),
            "quantize launch");
    return MOE_OK;
}

moe_status_t moe_dequantize_rows(int32_t fmt, const void *codes, const void *scales, int64_t rows, int32_t cols,
                                 const float *globals, int64_t per, int32_t type, void *dst, int64_t stride,
                                 void *stream) {
    RowsParams p;
    moe_status_t st = check_rows(fmt, type, dst, stride, rows, cols, globals, per, codes, scales, p);
    if (st != MOE_OK) return st;
    HIP_TRY(launch_dequantize(fmt, type, p, static_cast<const uint8_t *>(codes),
                              static_cast<const uint8_t *>(scales), dst, static_cast<hipStream_t>(stream)),
            "dequantize launch");
    return MOE_OK;
}

int64_t moe_mx_product_workspace_bytes(int32_t P, int32_t n, int32_t k, int32_t T, int32_t K) {
    if (check_mx_sizes(P, n, k, T, K) != MOE_OK) return 0;
    return (int64_t)mx_workspace_bytes(P, n, k, T, K);
}

moe_status_t moe_mx_product(const moe_mx_bank_t *bank, const void *x, int64_t x_stride, const int32_t *idx,
                            int32_t T, int32_t K, int32_t swiglu, int32_t out_type, void *out, void *ws,
                            int64_t ws_bytes, void *stream) {
    if (!bank) return fail(MOE_INVALID_ARG, "bank is NULL");
    moe_status_t st = check_mx_sizes(bank->num_rows, bank->n, bank->k, T, K);
    if (st != MOE_OK) return st;
    if (swiglu != 0 && swiglu != 1) return fail(MOE_INVALID_ARG, "swiglu must be 0 or 1");
    if (swiglu && bank->n % 2) return fail(MOE_INVALID_ARG, "swiglu needs an even n, got %d", bank->n);
    if (!known_type(out_type)) return fail(MOE_INVALID_ARG, "unknown output type %d", out_type);
    if (x_stride < bank->k) return fail(MOE_INVALID_ARG, "x stride %lld < k=%d", (long long)x_stride, bank->k);
    if (!bank->codes_dev || !bank->scales_dev || !aligned16(bank->codes_dev))
        return fail(MOE_INVALID_ARG, "bank codes or scales are NULL, or the codes not 16-byte aligned");
    if (!idx && (bank->num_rows != 1 || K != 1))
        return fail(MOE_INVALID_ARG, "idx is NULL for %d matrices and K=%d", bank->num_rows, K);
    if (T == 0) return MOE_OK;
    if (!x || !out || !ws) return fail(MOE_INVALID_ARG, "NULL product buffer");
    if (reinterpret_cast<uintptr_t>(x) % 2 || reinterpret_cast<uintptr_t>(out) % type_bytes(out_type) ||
        reinterpret_cast<uintptr_t>(idx) % 4)
        return fail(MOE_INVALID_ARG, "product buffers are not aligned to their elements");
    if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(MOE_INVALID_ARG, "workspace must be 256-byte aligned");
    const size_t need = mx_workspace_bytes(bank->num_rows, bank->n, bank->k, T, K);
    if (ws_bytes < (int64_t)need)
        return fail(MOE_INVALID_ARG, "workspace %lld B < %zu B", (long long)ws_bytes, need);
    MxParams p{};
    p.codes = static_cast<const uint8_t *>(bank->codes_dev);
    p.scales = static_cast<const uint8_t *>(bank->scales_dev);
    p.P = bank->num_rows;
    p.n = bank->n;
    p.k = bank->k;
    p.x = static_cast<const uint16_t *>(x);
    p.x_stride = x_stride;
    p.idx = idx;
    p.T = T;
    p.K = K;
    p.swiglu = swiglu;
    p.out_type = out_type;
    p.out = out;
    p.ws = static_cast<uint8_t *>(ws);
    if (!mx_launchable(p)) return fail(MOE_UNSUPPORTED, "%d routes of %d x %d: too many tiles", T * K, p.n, p.k);
    int lists = 0;
    HIP_TRY(launch_mx_product(p, &lists, static_cast<hipStream_t>(stream)), "MXFP4 product launch");
    return MOE_OK;
}

int64_t moe_routed_mx_workspace_bytes(int32_t P, int32_t H, int32_t F, int32_t T, int32_t K) {
    if (check_routed_mx_sizes(P, H, F, T, K) != MOE_OK) return 0;
    return (int64_t)routed_mx_ws(P, H, F, T, K).total;
}

moe_status_t moe_routed_decode_mx(const moe_pool_t *pool, const void *x, const int32_t *idx, const float *w,
                                  int32_t T, int32_t K, const float *addend, void *out, void *ws,
                                  int64_t ws_bytes, void *stream) {
    if (!pool) return fail(MOE_INVALID_ARG, "pool is NULL");
    if (pool->weight_format != MOE_FMT_MXFP4)
        return fail(MOE_INVALID_ARG, "weight format %d: 4-bit activations need an MXFP4 pool", pool->weight_format);
    const int P = pool->num_rows, H = pool->hidden, F = pool->ffn;
    moe_status_t st = check_routed_mx_sizes(P, H, F, T, K);
    if (st != MOE_OK) return st;
    for (int b = 0; b < bank_count(MOE_FMT_MXFP4); ++b)
        if (!pool->banks_dev[b] || (b % 2 == 0 && !aligned16(pool->banks_dev[b])))
            return fail(MOE_INVALID_ARG, "pool bank %d is NULL or not 16-byte aligned", b);
    if (T == 0) return MOE_OK;
    if (!x || !idx || !w || !out || !ws) return fail(MOE_INVALID_ARG, "NULL routed buffer");
    if (!aligned16(x)) return fail(MOE_INVALID_ARG, "x must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(idx) % 4 || reinterpret_cast<uintptr_t>(w) % 4 ||
        reinterpret_cast<uintptr_t>(addend) % 4 || reinterpret_cast<uintptr_t>(out) % 2)
        return fail(MOE_INVALID_ARG, "routed buffers are not aligned to their elements");
    if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(MOE_INVALID_ARG, "workspace must be 256-byte aligned");
    const RoutedMxWs L = routed_mx_ws(P, H, F, T, K);
    if (ws_bytes < (int64_t)L.total)
        return fail(MOE_INVALID_ARG, "workspace %lld B < %zu B", (long long)ws_bytes, L.total);
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *base = static_cast<uint8_t *>(ws);
    uint16_t *h = reinterpret_cast<uint16_t *>(base + L.h);
    float *d = reinterpret_cast<float *>(base + L.d);
    MxParams up{}, down{};
    up.codes = static_cast<const uint8_t *>(pool->banks_dev[0]);
    up.scales = static_cast<const uint8_t *>(pool->banks_dev[1]);
    up.P = P;
    up.n = 2 * F;
    up.k = H;
    up.x = static_cast<const uint16_t *>(x);
    up.x_stride = H;
    up.idx = idx;
    up.T = T;
    up.K = K;
    up.swiglu = 1;
    up.out_type = MOE_TYPE_BF16;
    up.out = h;
    up.ws = base;
    down = up;
    down.codes = static_cast<const uint8_t *>(pool->banks_dev[2]);
    down.scales = static_cast<const uint8_t *>(pool->banks_dev[3]);
    down.n = H;
    down.k = F;
    down.x = h;
    down.x_stride = F;
    down.T = T * K;   // a row of h for each route
    down.K = 1;
    down.swiglu = 0;
    down.out_type = MOE_TYPE_F32;
    down.out = d;
    if (!mx_launchable(up) || !mx_launchable(down))
        return fail(MOE_UNSUPPORTED, "%d routes of hidden %d, ffn %d: too many tiles", T * K, H, F);
    int lists = 0;
    HIP_TRY(launch_mx_product(up, &lists, s), "gate/up product launch");
    HIP_TRY(launch_mx_product(down, &lists, s), "down product launch");
    HIP_TRY(launch_combine(idx, w, T, K, H, P, d, addend, static_cast<uint16_t *>(out), s), "combine launch");
    return MOE_OK;
}

}  // extern "C"
