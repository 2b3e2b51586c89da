// Scored top-K routing: one wavefront per token row.
//
// For a row of logits l: scores s (softmax or sigmoid), choice values
// c = s + bias, groups ranked by their best or two best c, the K largest c
// of the kept groups, weights s renormalised and scaled.  Ties go to the
// lower index, and two scores that differ by less than an fp32 rounding are
// still two scores: they are computed and compared in 64 bits.
//
// A lane holds experts lane, lane + 64, ... of the row.  A choice value is
// kept as a 64-bit integer whose unsigned order is the order of the values
// (0: not available), split into its halves: a selection round takes the
// wave's maximum of the upper halves alone (DPP max steps) and looks at the
// lower halves and the index only where two candidates share it.  Lane k
// keeps pick k and recomputes its score at the end, so no score is carried
// through the rounds.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kRowsPerBlock = 4;

// Order-preserving image of a double (never 0 for a number above -infinity).
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);   // -0 counts as 0
    return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __longlong_as_double((long long)(k ^ ((k >> 63) ? 0x8000000000000000ull : ~0ull)));
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
    return v;
}

__device__ __forceinline__ float load_logit(const float *p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t *p) { return bf16_f(*p); }

// exp(l - top) of an available logit; the row's largest is 1 also where it
// is +infinity.
__device__ __forceinline__ double shifted_exp(float l, float top) {
    return l == top ? 1.0 : exp((double)l - (double)top);
}
__device__ __forceinline__ double sigmoid(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

// The two largest of two sorted pairs (0 = none).
__device__ __forceinline__ void merge_top2(uint64_t &a, uint64_t &b, uint64_t oa, uint64_t ob) {
    const uint64_t lo = a < oa ? a : oa;
    a = a < oa ? oa : a;
    b = b < ob ? ob : b;
    b = b < lo ? lo : b;
}

template <int VPL, typename L>
__global__ __launch_bounds__(kRowsPerBlock *kWave) void route_kernel(
    const L *__restrict__ logits, int64_t stride, int T, int E, int K, RouteParams p,
    int32_t *__restrict__ ids, float *__restrict__ w) {
    extern __shared__ __align__(16) uint64_t keys_lds[];   // [rows per block][E], groups only
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int row = blockIdx.x * kRowsPerBlock + wave;
    if (row >= T) return;
    const L *lr = logits + (int64_t)row * stride;

    float v[VPL];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = lane + kWave * j;
        const float l = e < E ? load_logit(lr + e) : -INFINITY;
        v[j] = l != l ? -INFINITY : l;
        top = fmaxf(top, v[j]);
    }
    // Scores are needed for every expert where the choice adds a bias or
    // sums two of a group; a plain softmax weight needs their sum too.
    const bool softmax = p.score == MOE_SCORE_SOFTMAX;
    const bool score_keys = p.bias != nullptr || (p.num_groups > 1 && p.group_score == MOE_GROUP_TOP2);
    double z = 1.0;
    if (softmax) {
        top = wave_max(top);
        if (score_keys || !p.renormalize) {
            double part = 0.0;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (v[j] > -INFINITY) part += shifted_exp(v[j], top);
            z = wave_sum(part);
        }
    }
    auto score_of = [&](float l) { return softmax ? shifted_exp(l, top) / z : sigmoid(l); };

    // choice keys; with groups ranked by score sums and no bias, the group
    // keys (scores) differ from the choice keys (logits)
    uint32_t hi[VPL], lo[VPL];
    uint64_t *gk = keys_lds + (size_t)wave * E;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = lane + kWave * j;
        uint64_t key = 0, gkey = 0;
        if (v[j] > -INFINITY) {
            double c = (double)v[j];
            if (score_keys) {
                const double s = score_of(v[j]);
                gkey = order_key(s);
                if (p.bias != nullptr) {
                    c = s + (double)p.bias[e];
                    gkey = c > -INFINITY ? order_key(c) : 0;
                }
            }
            key = c > -INFINITY ? order_key(c) : 0;
            if (!score_keys) gkey = key;
        }
        if (p.num_groups > 1 && e < E) gk[e] = gkey;
        hi[j] = (uint32_t)(key >> 32);
        lo[j] = (uint32_t)key;
    }

    if (p.num_groups > 1) {
        // 64 / 2^ceil(log2 G) lanes scan each group, then pair up
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int G = p.num_groups, gs = E / G;
        const int lanes = kWave >> p.log_groups;
        const int g = lane / lanes, sub = lane & (lanes - 1);
        uint64_t a = 0, b = 0;
        if (g < G)
            for (int i = sub; i < gs; i += lanes) {
                const uint64_t k = gk[g * gs + i];
                merge_top2(a, b, k, 0);
            }
        for (int off = 1; off < lanes; off <<= 1) {
            const uint64_t oa = __shfl_xor(a, off, kWave), ob = __shfl_xor(b, off, kWave);
            merge_top2(a, b, oa, ob);
        }
        uint64_t value = a;
        if (p.group_score == MOE_GROUP_TOP2 && b != 0) value = order_key(key_value(a) + key_value(b));
        // how many groups come before this one: larger, or equal and lower
        int before = 0;
        for (int og = 0; og < G; ++og) {
            const uint64_t ov = __shfl(value, og * lanes, kWave);
            before += ov > value || (ov == value && og < g);
        }
        const uint64_t kept = __ballot(g < G && value != 0 && before < p.top_groups);
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = lane + kWave * j;
            const int eg = gs == 1 ? e : (int)__umulhi((uint32_t)e, p.group_magic);   // e / gs
            if (e < E && !((kept >> (eg * lanes)) & 1)) hi[j] = lo[j] = 0;
        }
    }

    int mine = -1;
    for (int k = 0; k < K; ++k) {
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) best = max(best, hi[j]);
        const uint32_t m = wave_max_u32(best);
        if (m == 0) break;
        int at = -1, n = 0;
#pragma unroll
        for (int j = VPL - 1; j >= 0; --j)
            if (hi[j] == m) {
                at = j;
                ++n;
            }
        const uint64_t who = __ballot(n > 0);
        int e;
        if (__popcll(who) == 1 && __ballot(n > 1) == 0) {
            e = __builtin_amdgcn_readlane(lane + kWave * at, __ffsll((unsigned long long)who) - 1);
        } else {
            // equal upper halves: the larger lower half, then the lower index
            uint64_t t = 0;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (hi[j] == m) {
                    const uint64_t c = ((uint64_t)lo[j] << 32) | (uint32_t)~(lane + kWave * j);
                    t = c > t ? c : t;
                }
            t = wave_max_u64(t);
            e = (int)~(uint32_t)t;
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (lane + kWave * j == e) hi[j] = 0;
        if (lane == k) mine = e;
    }

    double s = 0.0;
    if (mine >= 0) s = score_of(load_logit(lr + mine));
    if (p.renormalize) {
        const double total = wave_sum(s);
        const int n = __popcll(__ballot(mine >= 0));
        s = total > 0.0 ? s / total : (mine >= 0 ? 1.0 / n : 0.0);
    }
    if (lane < K) {
        ids[(int64_t)row * K + lane] = mine;
        w[(int64_t)row * K + lane] = (float)(s * (double)p.scale);
    }
}

template <typename L>
hipError_t launch_route_typed(const L *logits, int64_t stride, int T, int E, int K, const RouteParams &p,
                              int32_t *ids, float *w, hipStream_t s) {
    const int blocks = (T + kRowsPerBlock - 1) / kRowsPerBlock;
    const size_t lds = p.num_groups > 1 ? (size_t)kRowsPerBlock * E * 8 : 0;   // at most 64 KB
    const int vpl = (E + kWave - 1) / kWave;
#define MOE_ROUTE(V)                                                                                       \
    hipLaunchKernelGGL((route_kernel<V, L>), dim3(blocks), dim3(kRowsPerBlock *kWave), lds, s, logits, stride, \
                       T, E, K, p, ids, w)
    if (vpl <= 1)
        MOE_ROUTE(1);
    else if (vpl <= 2)
        MOE_ROUTE(2);
    else if (vpl <= 4)
        MOE_ROUTE(4);
    else if (vpl <= 8)
        MOE_ROUTE(8);
    else if (vpl <= 16)
        MOE_ROUTE(16);
    else
        MOE_ROUTE(32);
#undef MOE_ROUTE
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteParams &p, int logits_type, const void *logits, int64_t stride, int T,
                        int E, int K, int32_t *ids, float *w, hipStream_t s) {
    if (T == 0) return hipSuccess;
    if (rec::on())
        return rec::launch("route_kernel", s, {{logits, rec::kRead}, {ids, rec::kWrite}, {w, rec::kWrite}});
    if (logits_type == MOE_TYPE_BF16)
        return launch_route_typed(static_cast<const uint16_t *>(logits), stride, T, E, K, p, ids, w, s);
    return launch_route_typed(static_cast<const float *>(logits), stride, T, E, K, p, ids, w, s);
}

}  // namespace moe
