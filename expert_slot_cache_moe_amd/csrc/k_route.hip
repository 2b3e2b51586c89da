// Scored top-K routing: one wavefront per token row.
//
// For a row of logits l: scores s (softmax or sigmoid), choice values
// c = s + bias, groups ranked by their best or two best c, the K largest c
// of the kept groups, weights s renormalised and scaled.  Ties go to the
// lower index, and two scores that differ by less than an fp32 rounding are
// still two scores: they are computed and compared in 64 bits.
//
// A lane holds experts lane, lane + 64, ... of the row.  Choice values are
// first formed in fp32, where their error is bounded; the K-th largest of
// the 64 lanes' own maxima, less that bound, is a floor that every pick
// reaches and few others do.  The candidates are packed one to a lane, their
// values computed in 64 bits, and their ranks counted.  Where more than 64
// values reach the floor (rows of equal scores), or two groups at the border
// of the choice are closer than the bound, the row takes the long way: every
// value in 64 bits, K rounds of a wave maximum.
//
// On MI355X one row of 256 grouped experts takes 4.8 us, the latency of its
// steps one behind the other; 16384 rows of 512 (33.5 MB) 22 us, where
// reading them takes 7.  What a row waits for shows in the built code: each
// of its eight values loads its bias on a branch and waits for it there, and
// the kind of score, the bias and the groups are branches of every value;
// what of the 22 us each part costs has not been counted.  The long way for
// every row took 95.  Four rows to a wave, whose serial parts overlap but
// whose registers allow fewer waves, took 21.3 at 512 experts and 12.2 (one
// row: 10.8) at 256.
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

// Sum over the wave, to every lane, in a fixed order (DPP moves of the halves).
__device__ __forceinline__ double wave_total(double v) {
#define MOE_ADD_STEP(CTRL, RM)                                                                        \
    {                                                                                                 \
        const uint64_t u = (uint64_t)__double_as_longlong(v);                                         \
        const uint32_t l = dpp_or_zero<CTRL, RM>((uint32_t)u), h = dpp_or_zero<CTRL, RM>((uint32_t)(u >> 32)); \
        v += __longlong_as_double((long long)(((uint64_t)h << 32) | l));                              \
    }
    MOE_ADD_STEP(kDppRowShr1, 0xf)
    MOE_ADD_STEP(kDppRowShr2, 0xf)
    MOE_ADD_STEP(kDppRowShr4, 0xf)
    MOE_ADD_STEP(kDppRowShr8, 0xf)
    MOE_ADD_STEP(kDppRowBcast15, 0xa)
    MOE_ADD_STEP(kDppRowBcast31, 0xc)
#undef MOE_ADD_STEP
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t l = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, kWave - 1);
    const uint32_t h = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), kWave - 1);
    return __longlong_as_double((long long)(((uint64_t)h << 32) | l));
}

// Largest of v over the wave, to every lane.
__device__ __forceinline__ float wave_max_f32(float v) {
#define MOE_MAX_STEP(CTRL, RM)                                                                              \
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, RM, \
                                                            0xf, false)));
    MOE_MAX_STEP(kDppRowShr1, 0xf)
    MOE_MAX_STEP(kDppRowShr2, 0xf)
    MOE_MAX_STEP(kDppRowShr4, 0xf)
    MOE_MAX_STEP(kDppRowShr8, 0xf)
    MOE_MAX_STEP(kDppRowBcast15, 0xa)
    MOE_MAX_STEP(kDppRowBcast31, 0xc)
#undef MOE_MAX_STEP
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), kWave - 1));
}

// What one row needs, in registers and in the wave's LDS.
template <int VPL> struct RowState {
    float v[VPL];         // logits, -infinity where there is none
    float top;            // softmax: the largest
    double z;             // softmax: sum of exp(l - top), or 1 where it is not needed
    const RouteParams &p;
    __device__ __forceinline__ double score(float l) const {
        return p.score == MOE_SCORE_SOFTMAX ? shifted_exp(l, top) / z : sigmoid(l);
    }
    // what experts are picked by; -infinity: not available
    __device__ __forceinline__ double choice(float l, int e) const {
        if (!(l > -INFINITY)) return -INFINITY;
        const double c = p.bias != nullptr ? score(l) + (double)p.bias[e] : (double)l;
        return c > -INFINITY ? c : -INFINITY;   // NaN too
    }
};

struct Candidate {
    float l;
    int32_t e;
};
// The floor may let through this many lanes more than K, and is looked for
// by at most so many halvings.
constexpr int kSpare = 4, kHalvings = 10;

// The wave's lanes g * lanes .. of group g; every group's place among the
// groups, by `before`.
template <typename V> __device__ __forceinline__ uint64_t kept_groups(const RouteParams &p, int lane, V value, V none) {
    const int lanes = kWave >> p.log_groups, g = lane / lanes;
    int before = 0;
    for (int og = 0; og < p.num_groups; ++og) {
        const V ov = __shfl(value, og * lanes, kWave);
        before += ov > value || (ov == value && og < g);
    }
    return __ballot(g < p.num_groups && value != none && before < p.top_groups);
}

// e / (E / G) by multiplication.
__device__ __forceinline__ int group_of(const RouteParams &p, int gs, int e) {
    return gs == 1 ? e : (int)__umulhi((uint32_t)e, p.group_magic);
}

__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The long way: every choice value in 64 bits, as integers of the same
// order (0: not available), K rounds of a maximum of their upper halves.
// Returns lane k's pick k, or -1.
template <int VPL>
__device__ __forceinline__ int pick_long_way(const RowState<VPL> &row, const RouteParams &p, int E, int K,
                                                       int lane, uint64_t *gk) {
    uint32_t hi[VPL], lo[VPL];
    const bool score_sums = p.num_groups > 1 && p.group_score == MOE_GROUP_TOP2 && p.bias == nullptr;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = lane + kWave * j;
        const double c = e < E ? row.choice(row.v[j], e) : -INFINITY;
        const uint64_t key = c > -INFINITY ? order_key(c) : 0;
        if (p.num_groups > 1 && e < E) gk[e] = key != 0 && score_sums ? order_key(row.score(row.v[j])) : key;
        hi[j] = (uint32_t)(key >> 32);
        lo[j] = (uint32_t)key;
    }
    if (p.num_groups > 1) {
        wave_lds_sync();
        const int G = p.num_groups, gs = E / G;
        const int lanes = kWave >> p.log_groups, g = lane / lanes;
        uint64_t a = 0, b = 0;
        if (g < G)
            for (int i = lane & (lanes - 1); i < gs; i += lanes) merge_top2(a, b, gk[g * gs + i], (uint64_t)0);
        for (int off = 1; off < lanes; off <<= 1) {
            const uint64_t oa = __shfl_xor(a, off, kWave), ob = __shfl_xor(b, off, kWave);
            merge_top2(a, b, oa, ob);
        }
        uint64_t value = a;
        if (p.group_score == MOE_GROUP_TOP2 && b != 0) value = order_key(key_value(a) + key_value(b));
        const uint64_t kept = kept_groups<uint64_t>(p, lane, value, 0);
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = lane + kWave * j;
            if (e < E && !((kept >> (group_of(p, gs, e) * lanes)) & 1)) hi[j] = lo[j] = 0;
        }
    }
    int mine = -1;
    for (int k = 0; k < K; ++k) {
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) best = max(best, hi[j]);
        const uint32_t m = wave_max_u32(best);
        if (m == 0) break;
        // among equal upper halves the larger lower half, then the lower index
        uint64_t t = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (hi[j] == m) {
                const uint64_t c = ((uint64_t)lo[j] << 32) | (uint32_t)~(lane + kWave * j);
                t = c > t ? c : t;
            }
        const int e = (int)~(uint32_t)wave_max_u64(t);
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (lane + kWave * j == e) hi[j] = 0;
        if (lane == k) mine = e;
    }
    return mine;
}

template <int VPL, typename L>
__global__ __launch_bounds__(kRowsPerBlock *kWave) void route_kernel(
    const L *__restrict__ logits, int64_t stride, int T, int E, int K, RouteParams p,
    int32_t *__restrict__ ids, float *__restrict__ w) {
    extern __shared__ __align__(16) uint64_t lds[];   // [rows per block][E], groups only
    __shared__ Candidate cand[kRowsPerBlock][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int row_i = blockIdx.x * kRowsPerBlock + wave;
    if (row_i >= T) return;
    const L *lr = logits + (int64_t)row_i * stride;

    RowState<VPL> row{{}, -INFINITY, 1.0, p};
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = lane + kWave * j;
        const float l = e < E ? load_logit(lr + e) : -INFINITY;
        row.v[j] = l != l ? -INFINITY : l;
        row.top = fmaxf(row.top, row.v[j]);
    }
    const bool softmax = p.score == MOE_SCORE_SOFTMAX, biased = p.bias != nullptr;
    const bool top2 = p.num_groups > 1 && p.group_score == MOE_GROUP_TOP2;
    if (softmax) {
        row.top = wave_max_f32(row.top);
        // a renormalised softmax weight needs no sum over the row, and
        // neither does the order without a bias
        if (biased || !p.renormalize) {
            double part = 0.0;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (row.v[j] > -INFINITY) part += shifted_exp(row.v[j], row.top);
            row.z = wave_total(part);
        }
    }

    // Choice values in fp32.  exp and the reciprocal are good to a few ulp,
    // and an error d in their argument l shows as |l| s (1 - s) 2^-24 in the
    // score: scores are within 2^-21, their sums with a bias within 2^-21 +
    // 2^-24 |c|.  Two values further apart than slack(c) are in true order.
    auto slack = [](float c) { return (1.f + fabsf(c)) * 0x1p-19f; };
    const float rz = (float)(1.0 / row.z);
    auto score32 = [&](float l) {
        if (softmax) return l == row.top ? rz : expf(l - row.top) * rz;
        return __builtin_amdgcn_rcpf(1.f + __expf(-l));
    };
    float c[VPL], gv[VPL];   // choice and, for the groups, what their value is made of
    float best = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = lane + kWave * j;
        const bool on = row.v[j] > -INFINITY;
        float s = 0.f;
        if (biased || top2) s = score32(row.v[j]);
        c[j] = row.v[j];
        if (biased) c[j] = s + (e < E ? p.bias[e] : 0.f);
        c[j] = on && c[j] > -INFINITY ? c[j] : -INFINITY;
        gv[j] = top2 && !biased && on ? s : c[j];
    }

    bool settled = true;
    if (p.num_groups > 1) {
        float *gl = reinterpret_cast<float *>(lds + (size_t)wave * E);
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (lane + kWave * j < E) gl[lane + kWave * j] = gv[j];
        wave_lds_sync();
        const int G = p.num_groups, gs = E / G;
        const int lanes = kWave >> p.log_groups, g = lane / lanes;
        float a = -INFINITY, b = -INFINITY;
        auto merge = [&](float oa, float ob) {
            const float lo = fminf(a, oa);
            a = fmaxf(a, oa);
            b = fmaxf(fmaxf(b, ob), lo);
        };
        if (g < G)
            for (int i = lane & (lanes - 1); i < gs; i += lanes) merge(gl[g * gs + i], -INFINITY);
        for (int off = 1; off < lanes; off <<= 1) {
            const float oa = __shfl_xor(a, off, kWave), ob = __shfl_xor(b, off, kWave);
            merge(oa, ob);
        }
        const float value = top2 && b > -INFINITY ? a + b : a;
        const uint64_t kept = kept_groups<float>(p, lane, value, -INFINITY);
        if (biased || top2) {
            // the kept and the dropped must be further apart than their errors
            const bool in = (kept >> lane) & 1;
            const float err = slack(a) + (top2 && b > -INFINITY ? slack(b) : 0.f);
            const float under = err < INFINITY ? value - err : -INFINITY, over = err < INFINITY ? value + err : INFINITY;
            const float worst = -wave_max_f32(in ? -under : -INFINITY);
            const float next = wave_max_f32(g < G && !in && value > -INFINITY ? over : -INFINITY);
            settled = worst > next || !(next > -INFINITY);
            // two values of the lowest kind (experts biased out of reach, but
            // available) add up to -infinity in fp32, not in 64 bits
            if (top2) settled = settled && __ballot(b > -INFINITY && !(value > -INFINITY)) == 0;
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = lane + kWave * j;
            if (e < E && !((kept >> (group_of(p, gs, e) * lanes)) & 1)) c[j] = -INFINITY;
        }
        wave_lds_sync();   // the long way writes the same LDS
    }

    // The floor: a value that at least K, and not many more, of the lanes'
    // maxima reach -- found by halving the range between their least and
    // largest, or, where that has not narrowed it (maxima many magnitudes
    // apart), as the K-th largest maximum itself.
#pragma unroll
    for (int j = 0; j < VPL; ++j) best = fmaxf(best, c[j]);
    float low = -INFINITY;
    if (VPL > 1 && __popcll(__ballot(best > -INFINITY)) > K + kSpare) {
        float under = -wave_max_f32(best > -INFINITY ? -best : -INFINITY), over = wave_max_f32(best);
        int n = kWave;
        for (int i = 0; i < kHalvings && n > K + kSpare; ++i) {
            const float mid = 0.5f * under + 0.5f * over;
            const int m = __popcll(__ballot(best >= mid));
            if (m >= K) {
                under = mid;
                n = m;
            } else {
                over = mid;
            }
        }
        low = under;
        if (n > kWave / 2) {
            n = 0;
            while (n < K) {
                low = wave_max_f32(best);
                const bool is = best == low;
                n += __popcll(__ballot(is));
                if (is) best = -INFINITY;
            }
        }
        if (biased) low -= slack(low);
        if (!(low > -INFINITY)) low = -INFINITY;   // also where it is NaN: infinity less infinity
    }
    int n = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const bool in = c[j] > -INFINITY && c[j] >= low;
        const uint64_t m = __ballot(in);
        const int at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
        if (in && at < kWave) cand[wave][at] = Candidate{row.v[j], lane + kWave * j};
        n += __popcll(m);
    }
    settled = settled && n <= kWave;

    int rank = lane;      // the place of this lane's pick
    Candidate my{-INFINITY, -1};
    double s = 0.0;       // its score
    if (settled) {
        wave_lds_sync();
        if (lane < n) my = cand[wave][lane];
        // candidates lie in index order: of equal values the lower lane is first
        rank = 0;
        if (biased) {
            s = row.score(my.l);
            const double mine = lane < n ? s + (double)p.bias[my.e] : -INFINITY;
            const uint64_t key = order_key(mine);
            for (int i = 0; i < n; ++i) {
                const uint64_t ok =
                    ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(key >> 32), i) << 32) |
                    (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, i);
                rank += ok > key || (ok == key && i < lane);
            }
        } else {
            for (int i = 0; i < n; ++i) {
                const float ol = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my.l), i));
                rank += ol > my.l || (ol == my.l && i < lane);
            }
            s = row.score(my.l);
        }
        if (lane >= n) rank = lane;   // behind the candidates
    } else {
        my.e = pick_long_way<VPL>(row, p, E, K, lane, lds + (size_t)wave * E);
        if (my.e >= 0) s = row.score(load_logit(lr + my.e));
    }

    const bool picked = my.e >= 0 && rank < K;
    if (!picked) s = 0.0;
    if (p.renormalize) {
        const double total = wave_total(s);
        const int count = __popcll(__ballot(picked));
        s = total > 0.0 ? s / total : (picked ? 1.0 / count : 0.0);
    }
    if (rank < K) {
        ids[(int64_t)row_i * K + rank] = picked ? my.e : -1;
        w[(int64_t)row_i * K + rank] = (float)(s * (double)p.scale);
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
