// Rows of floats to the 4-bit bank formats, and back.
//
// One pass: an MXFP4 lane holds 8 consecutive elements, and the 4 lanes of a
// block share their largest magnitude; an E2M1 lane holds a block of 16.
//
// MXFP4 scales are powers of two, so x / scale is exact and rounded once, by
// the hardware's scaled conversion.  E2M1 scales are not: x / (scale g) is
// rounded wherever it is formed, and a value next to the middle of two codes
// could cross it.  The middles m scale g have at most 31 significant bits (m
// 3, scale 4, g 24) and x at most 24, so a quotient that is not exactly a
// middle differs from it by more than 2^-32 of its size.  A quotient of two
// fp32 parts tells the two apart; it is handed to the conversion rounded to
// odd, which keeps what lies off a middle off it.  The same holds for the
// scale itself, a / (6 g) against the middles of E4M3.
//
// Bound by memory: a 134M element bf16 matrix (340 MB of both sides) to
// MXFP4 and back takes 133 us on MI355X (5.1 TB/s; a large copy reaches
// 4.9); to E2M1 and back 144, the way there 78 to 82 of them, bound by the
// quotients.  One row of 2048 takes 1.4 us either way, less than its launch.
#include "k_rows.inc"

namespace moe {
namespace {

using namespace rows_detail;

constexpr int kThreads = 256;

// ---- any g: quotients in 64 bits

// x inv to fp32 for the E2M1 conversion: cut to 24 bits, with the last bit
// set where more was cut than the quotient's own error.  inv carries a
// factor 1 + 2^-50, above every rounding in it (3 x 2^-53), so an exact
// middle lands on itself and up to 2^-49 above, never below; the tail below
// 2^-44 counts as nothing.
__device__ __forceinline__ float quotient64(float x, double inv) {
    const double y = (double)x * inv;
    uint64_t u = (uint64_t)__double_as_longlong(y);
    const uint32_t tail = (uint32_t)u & 0x1fffffffu;   // the 29 bits below fp32's last
    u &= ~0x1fffffffull;
    if (tail >= (1u << 8)) u |= 0x20000000u;
    return __builtin_amdgcn_fmed3f((float)__longlong_as_double((long long)u), -8.f, 8.f);
}

// E4M3 byte of v >= 0: nearest, ties to even, at most 448.
__device__ __forceinline__ uint32_t e4m3_of(double v) {
    if (v >= 448.0) return 0x7E;
    int e = v >= 0x1p-6 ? ilogb(v) : -6;
    const double q = rint(ldexp(v, 3 - e));   // 8..16 (0..8 subnormal)
    // a carry to 16 is the next exponent's 8
    return (uint32_t)((e + 6) * 8 + (int)q);
}

// ---- g of ordinary size (2^-80 to 2^80): the same in pairs of fp32, which
// took the 134M element matrix from 127 to 79 us

// E4M3 byte of a / (6 g): a candidate from an approximate quotient, moved up
// where a lies above the middle over it (or on it, and the candidate is
// odd).  6 g = hi + lo exactly, and a - middle hi is exact wherever it is
// small enough for middle lo to matter, so the comparison is exact.
__device__ __forceinline__ uint32_t e4m3_of(float a, float g) {
    const float hi = 6.f * g, lo = fmaf(6.f, g, -hi);
    const float t = a * __builtin_amdgcn_rcpf(hi);
    if (t >= 470.f) return 0x7E;
    const int e = max((int)(__float_as_uint(t) >> 23) - 127, -6);
    const int k = (int)floorf(ldexpf(t, 3 - e));
    const float middle = ldexpf((float)k + 0.5f, e - 3);
    const float over = fmaf(-middle, lo, fmaf(-middle, hi, a));
    const int q = k + (over > 0.f || (over == 0.f && (k & 1)));
    return (uint32_t)min((e + 6) * 8 + q, 0x7E);
}

// The reciprocal of u = s g (a scale of 4 bits, g of 24) in two parts.  TRIM:
// the first part has 16 bits, so that its product with a bf16 number is
// exact.  limit: a power of two of 8 u to 16 u.
template <bool TRIM>
__device__ __forceinline__ void reciprocal(float s, float g, float &ih, float &il, float &limit) {
    const float uh = s * g, ul = fmaf(s, g, -uh);
    limit = __uint_as_float((__float_as_uint(uh) & 0x7f800000u) + (4u << 23));
    float r = __builtin_amdgcn_rcpf(uh);
    r = fmaf(r, fmaf(-uh, r, 1.f), r);
    ih = TRIM ? __uint_as_float(__float_as_uint(r) & 0xffffff00u) : r;
    il = fmaf(-ul, ih, fmaf(-uh, ih, 1.f)) * r;
}

// x (ih + il) rounded to odd: the nearest fp32 p, its last bit set (and one
// taken off first, where the quotient is smaller) unless the rest is none.
// The two parts are good to 2^-39 of a quotient, of at most 5 where it
// matters: on a middle the rest is below 2^-36, and what is off a middle is
// off by at least 2^-33; 2^-35 tells them apart.
// A block whose scale stops at 448 may hold any x: what passes the limit is
// taken as the limit, a quotient above 8 where the largest code is 6.  (Cut
// behind the first product instead, x il would still grow with x, and il has
// either sign.)  The median, as fminf would first quiet a NaN in an
// instruction of its own.
template <bool TRIM> __device__ __forceinline__ float quotient(float x, float ih, float il, float limit) {
    const float ax = __builtin_amdgcn_fmed3f(fabsf(x), 0.f, limit);
    float p = ax * ih, rest;
    if constexpr (TRIM) {
        const float p0 = p;                   // exact
        p = fmaf(ax, il, p0);
        rest = fmaf(ax, il, p0 - p);
    } else {
        const float p0 = p, r0 = fmaf(ax, il, fmaf(ax, ih, -p0));
        p = p0 + r0;
        rest = r0 - (p - p0);
    }
    const uint32_t u = __float_as_uint(p);
    const uint32_t odd = (u + (uint32_t)((int)__float_as_uint(rest) >> 31)) | 1u;
    const uint32_t v = fabsf(rest) > 0x1p-35f ? odd : u;
    // (x ih may vanish and leave p the sign of x il)
    return copysignf(__uint_as_float(v), x);
}

// MXFP4: eight elements a lane.
template <bool VEC, typename SRC>
__global__ __launch_bounds__(kThreads) void quantize_mx_kernel(const SRC *__restrict__ src, int64_t stride,
                                                               int64_t units, int upr, FastDiv by_upr,
                                                               uint8_t *__restrict__ codes,
                                                               uint8_t *__restrict__ scales) {
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
        const int64_t row = (int64_t)by_upr((uint64_t)u);
        float f[kPer];
        load8<VEC>(src + row * stride + (u - row * upr) * kPer, f);
        uint32_t sc;
        const uint32_t c = mx_codes(f, quad_max(amax_bits(f)), sc);
        reinterpret_cast<uint32_t *>(codes)[u] = c;
        if ((threadIdx.x & 3) == 0) scales[u / 4] = (uint8_t)sc;
    }
}

// E2M1: a block of 16 a lane, so that its scale and reciprocal are made once.
template <bool VEC, typename SRC>
__global__ __launch_bounds__(kThreads) void quantize_e2m1_kernel(const SRC *__restrict__ src, int64_t stride,
                                                                 int64_t units, int upr, FastDiv by_upr,
                                                                 const float *__restrict__ globals,
                                                                 FastDiv by_global, uint8_t *__restrict__ codes,
                                                                 uint8_t *__restrict__ scales) {
    constexpr bool kTrim = sizeof(SRC) == 2;
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
        const int64_t row = (int64_t)by_upr((uint64_t)u);
        const SRC *p = src + row * stride + (u - row * upr) * 2 * kPer;
        float f[2][kPer];
        load8<VEC>(p, f[0]);
        load8<VEC>(p + kPer, f[1]);
        const float g = globals ? globals[by_global((uint64_t)row)] : 1.f;
        const uint32_t a = max(amax_bits(f[0]), amax_bits(f[1]));
        bool bad = a >= 0x7f800000u || !(g > 0.f && g < INFINITY);
        uint32_t sc;
        float q[2][kPer];
        if (g >= 0x1p-80f && g <= 0x1p80f) {
            sc = bad ? 0x7Fu : e4m3_of(__uint_as_float(a), g);
            float ih, il, limit;
            reciprocal<kTrim>(e4m3_f(sc), g, ih, il, limit);
#pragma unroll
            for (int i = 0; i < 2 * kPer; ++i)
                q[i / kPer][i % kPer] = quotient<kTrim>(f[i / kPer][i % kPer], ih, il, limit);
        } else {
            sc = bad ? 0x7Fu : e4m3_of((double)__uint_as_float(a) / (6.0 * (double)g));
            const double inv = 1.0 / ((double)e4m3_f(sc) * (double)g) * (1.0 + 0x1p-50);
#pragma unroll
            for (int i = 0; i < 2 * kPer; ++i) q[i / kPer][i % kPer] = quotient64(f[i / kPer][i % kPer], inv);
        }
        bad |= sc == 0;   // scale 0: codes 0
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#define MOE_CVT(B) c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[i], q[i][2 * B], q[i][2 * B + 1], 1.0f, B);
            MOE_CVT(0)
            MOE_CVT(1)
            MOE_CVT(2)
            MOE_CVT(3)
#undef MOE_CVT
        }
        reinterpret_cast<uint2 *>(codes)[u] = bad ? uint2{0, 0} : uint2{c[0], c[1]};
        scales[u] = (uint8_t)sc;
    }
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two products a g rounded once to bf16: the fp32 product rounded first
// could land on a bf16 middle that it is not on; its error (in 64 bits: of a
// product below 2^-126 it has bits under fp32's last) then says to which side
// it belongs.
__device__ __forceinline__ bool on_middle(float p) { return (__float_as_uint(p) & 0xffffu) == 0x8000u; }
__device__ __forceinline__ float off_middle(float a, float g) {
    const float p = a * g;
    uint32_t u = __float_as_uint(p);
    if (on_middle(p)) {
        const double err = (double)a * (double)g - (double)p;
        if (err != 0.0) u += ((err > 0.0) == (p > 0.f)) ? 1 : -1;
    }
    return __uint_as_float(u);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Back: a lane holds 8 MXFP4 codes, or a block of 16 E2M1 ones.
template <int FMT, bool VEC, typename DST>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales,
                                                              int64_t units, int upr, FastDiv by_upr,
                                                              const float *__restrict__ globals,
                                                              FastDiv by_global, DST *__restrict__ dst,
                                                              int64_t stride) {
    constexpr int kWords = FMT == MOE_FMT_MXFP4 ? 1 : 2, kN = 8 * kWords;
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
        const int64_t row = (int64_t)by_upr((uint64_t)u);
        uint32_t c[kWords];
        if constexpr (kWords == 2) {
            const uint2 t = reinterpret_cast<const uint2 *>(codes)[u];
            c[0] = t.x;
            c[kWords - 1] = t.y;
        } else {
            c[0] = reinterpret_cast<const uint32_t *>(codes)[u];
        }
        const uint32_t sc = scales[FMT == MOE_FMT_MXFP4 ? u / 4 : u];
        const float s = FMT == MOE_FMT_MXFP4 ? e8m0_f(sc) : e4m3_f(sc);
        DST *o = dst + row * stride + (u - row * upr) * kN;
        f32x2 f[kN / 2];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
#define MOE_CVT(B) f[4 * i + B] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], 1.0f, B);
            MOE_CVT(0)
            MOE_CVT(1)
            MOE_CVT(2)
            MOE_CVT(3)
#undef MOE_CVT
        }
        const bool scaled = FMT == MOE_FMT_E2M1 && globals != nullptr;
        const float g = scaled ? globals[by_global((uint64_t)row)] : 1.f;
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) f[i] = f32x2{f[i].x * s, f[i].y * s};   // exact
        uint32_t v[sizeof(DST) == 4 ? kN : kN / 2];
        bool middle = false;
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            const f32x2 t = scaled ? f32x2{f[i].x * g, f[i].y * g} : f[i];
            if constexpr (sizeof(DST) == 4) {
                v[2 * i] = __float_as_uint(t.x);
                v[2 * i + 1] = __float_as_uint(t.y);
            } else {
                v[i] = bf16_pair(t.x, t.y);
                if (scaled) middle |= on_middle(t.x) | on_middle(t.y);
            }
        }
        if constexpr (sizeof(DST) == 2) {
            if (middle) {   // one product in 2^16
#pragma unroll
                for (int i = 0; i < kN / 2; ++i) v[i] = bf16_pair(off_middle(f[i].x, g), off_middle(f[i].y, g));
            }
        }
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < (int)(sizeof v / 16); ++i)
                reinterpret_cast<u32x4 *>(o)[i] = u32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        } else if constexpr (sizeof(DST) == 4) {
#pragma unroll
            for (int i = 0; i < kN; ++i) o[i] = __uint_as_float(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) o[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
        }
    }
}

// Workgroups for `units` lanes of work: a few per CU, the rest by striding.
int grid_for(int64_t units) {
    const int64_t blocks = (units + kThreads - 1) / kThreads;
    return (int)(blocks < 65536 ? blocks : 65536);
}

}  // namespace

hipError_t launch_quantize(int fmt, int type, const RowsParams &p, const void *src, uint8_t *codes,
                           uint8_t *scales, hipStream_t s) {
    if (p.rows == 0) return hipSuccess;
    const bool vec = vector_rows(src, p.stride, p.rows, type == MOE_TYPE_F32 ? 4 : 2);
    const int upr = p.cols / (fmt == MOE_FMT_MXFP4 ? kPer : 2 * kPer);
    const int64_t units = p.rows * upr;
    const FastDiv by_upr(upr, units), by_global(p.globals ? p.rows_per_global : 1, p.rows);
#define MOE_MX(V, S)                                                                                    \
    hipLaunchKernelGGL((quantize_mx_kernel<V, S>), dim3(grid_for(units)), dim3(kThreads), 0, s,        \
                       static_cast<const S *>(src), p.stride, units, upr, by_upr, codes, scales)
#define MOE_E2M1(V, S)                                                                                  \
    hipLaunchKernelGGL((quantize_e2m1_kernel<V, S>), dim3(grid_for(units)), dim3(kThreads), 0, s,      \
                       static_cast<const S *>(src), p.stride, units, upr, by_upr, p.globals, by_global, \
                       codes, scales)
#define MOE_QUANT(K)            \
    if (type == MOE_TYPE_F32) { \
        if (vec)                \
            K(true, float);     \
        else                    \
            K(false, float);    \
    } else {                    \
        if (vec)                \
            K(true, uint16_t);  \
        else                    \
            K(false, uint16_t); \
    }
    if (fmt == MOE_FMT_MXFP4) {
        MOE_QUANT(MOE_MX)
    } else {
        MOE_QUANT(MOE_E2M1)
    }
#undef MOE_QUANT
#undef MOE_E2M1
#undef MOE_MX
    return hipGetLastError();
}

hipError_t launch_dequantize(int fmt, int type, const RowsParams &p, const uint8_t *codes,
                             const uint8_t *scales, void *dst, hipStream_t s) {
    if (p.rows == 0) return hipSuccess;
    const int upr = p.cols / (fmt == MOE_FMT_MXFP4 ? kPer : 2 * kPer);
    const int64_t units = p.rows * upr;
    const bool vec = vector_rows(dst, p.stride, p.rows, type == MOE_TYPE_F32 ? 4 : 2);
    const FastDiv by_upr(upr, units), by_global(p.globals ? p.rows_per_global : 1, p.rows);
#define MOE_DEQ(F, V, S)                                                                              \
    hipLaunchKernelGGL((dequantize_kernel<F, V, S>), dim3(grid_for(units)), dim3(kThreads), 0, s,    \
                       codes, scales, units, upr, by_upr, p.globals, by_global, static_cast<S *>(dst), \
                       p.stride)
#define MOE_DEQ_V(F, S)       \
    if (vec)                  \
        MOE_DEQ(F, true, S);  \
    else                      \
        MOE_DEQ(F, false, S);
    if (fmt == MOE_FMT_MXFP4 && type == MOE_TYPE_F32) {
        MOE_DEQ_V(MOE_FMT_MXFP4, float)
    } else if (fmt == MOE_FMT_MXFP4) {
        MOE_DEQ_V(MOE_FMT_MXFP4, uint16_t)
    } else if (type == MOE_TYPE_F32) {
        MOE_DEQ_V(MOE_FMT_E2M1, float)
    } else {
        MOE_DEQ_V(MOE_FMT_E2M1, uint16_t)
    }
#undef MOE_DEQ_V
#undef MOE_DEQ
    return hipGetLastError();
}

}  // namespace moe
