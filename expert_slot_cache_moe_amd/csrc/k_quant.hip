// Rows of floats to the 4-bit bank formats, and back.
//
// One pass: a lane holds 8 consecutive elements, the 4 (MXFP4) or 2 (E2M1)
// lanes of a block share their largest magnitude, and each lane writes its 8
// codes as one dword.
//
// MXFP4 scales are powers of two, so x / scale is exact and rounded once, by
// the hardware's scaled conversion.  E2M1 scales are not: x / (scale g) is rounded wherever it
// is formed, and a value next to the middle of two codes could cross it.
// The middles m scale g have at most 31 significant bits (m 3, scale 4, g
// 24) and x at most 24, so a quotient that is not exactly a middle differs
// from it by more than 2^-32 of its size: a 53-bit quotient tells the two
// apart, and is handed to the conversion with its tail folded into the last
// fp32 bit.
#include "k_rows.inc"

namespace moe {
namespace {

using namespace rows_detail;

constexpr int kThreads = 256;
// x inv to fp32 for the E2M1 conversion: cut to 24 bits, with the last bit
// set where more was cut than the quotient's own error.  inv carries a
// factor 1 + 2^-50, above every rounding in it (3 x 2^-53), so an exact
// middle lands on itself and up to 2^-49 above, never below; the tail below
// 2^-44 counts as nothing.
__device__ __forceinline__ float quotient(float x, double inv) {
    const double y = (double)x * inv;
    uint64_t u = (uint64_t)__double_as_longlong(y);
    const uint32_t tail = (uint32_t)u & 0x1fffffffu;   // the 29 bits below fp32's last
    u &= ~0x1fffffffull;
    if (tail >= (1u << 8)) u |= 0x20000000u;
    return (float)__longlong_as_double((long long)u);
}

// E4M3 byte of v >= 0: nearest, ties to even, at most 448.
__device__ __forceinline__ uint32_t e4m3_of(double v) {
    if (v >= 448.0) return 0x7E;
    int e = v >= 0x1p-6 ? ilogb(v) : -6;
    const double q = rint(ldexp(v, 3 - e));   // 8..16 (0..8 subnormal)
    // a carry to 16 is the next exponent's 8
    return (uint32_t)((e + 6) * 8 + (int)q);
}

template <int FMT, bool VEC, typename SRC>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const SRC *__restrict__ src, int64_t stride,
                                                            int64_t units, int upr, FastDiv by_upr,
                                                            const float *__restrict__ globals,
                                                            FastDiv by_global, uint8_t *__restrict__ codes,
                                                            uint8_t *__restrict__ scales) {
    constexpr int kLanes = FMT == MOE_FMT_MXFP4 ? 4 : 2;   // lanes per block
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
        const int64_t row = (int64_t)by_upr((uint64_t)u);
        float f[kPer];
        load8<VEC>(src + row * stride + (u - row * upr) * kPer, f);
        uint32_t a = amax_bits(f), sc, c = 0;
        if constexpr (FMT == MOE_FMT_MXFP4) {
            c = mx_codes(f, quad_max(a), sc);
        } else {
            a = pair_max(a);
            const float g = globals ? globals[by_global((uint64_t)row)] : 1.f;
            bool bad = a >= 0x7f800000u || !(g > 0.f && g < INFINITY);
            sc = bad ? 0x7Fu : e4m3_of((double)__uint_as_float(a) / (6.0 * (double)g));
            bad |= sc == 0;   // scale 0: codes 0
            const double inv = bad ? 0.0 : 1.0 / ((double)e4m3_f(sc) * (double)g) * (1.0 + 0x1p-50);
            if (!bad) {
                float q[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) q[i] = __builtin_amdgcn_fmed3f(quotient(f[i], inv), -8.f, 8.f);
#define MOE_CVT(B) c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[2 * B], q[2 * B + 1], 1.0f, B);
                MOE_CVT(0)
                MOE_CVT(1)
                MOE_CVT(2)
                MOE_CVT(3)
#undef MOE_CVT
            }
        }
        reinterpret_cast<uint32_t *>(codes)[u] = c;
        if ((threadIdx.x & (kLanes - 1)) == 0) scales[u / kLanes] = (uint8_t)sc;
    }
}

// code * scale * g rounded once to bf16: the fp32 product rounded first
// could land on a bf16 middle it is not on; its error (exact, by fma) then
// says to which side it belongs.
__device__ __forceinline__ uint16_t bf16_once(float a, float g) {
    const float p = a * g;
    uint32_t u = __float_as_uint(p);
    if ((u & 0xffffu) == 0x8000u) {
        const float err = fmaf(a, g, -p);
        if (err != 0.f) u += ((err > 0.f) == (p > 0.f)) ? 1 : -1;
    }
    return f32_to_bf16(__uint_as_float(u));
}

template <int FMT, bool VEC, typename DST>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales,
                                                              int64_t units, int upr, FastDiv by_upr,
                                                              const float *__restrict__ globals,
                                                              FastDiv by_global, DST *__restrict__ dst,
                                                              int64_t stride) {
    constexpr int kLanes = FMT == MOE_FMT_MXFP4 ? 4 : 2;
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
        const int64_t row = (int64_t)by_upr((uint64_t)u);
        const uint32_t c = reinterpret_cast<const uint32_t *>(codes)[u];
        const uint32_t sc = scales[u / kLanes];
        const float s = FMT == MOE_FMT_MXFP4 ? e8m0_f(sc) : e4m3_f(sc);
        const float g = FMT == MOE_FMT_E2M1 && globals ? globals[by_global((uint64_t)row)] : 1.f;
        float f[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) f[i] = e2m1_f((c >> (4 * i)) & 15u) * s;   // exact
        DST *o = dst + row * stride + (u - row * upr) * kPer;
        if constexpr (sizeof(DST) == 4) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) f[i] *= g;
            if constexpr (VEC) {
                u32x4 a, b;
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = __float_as_uint(f[i]), b[i] = __float_as_uint(f[4 + i]);
                reinterpret_cast<u32x4 *>(o)[0] = a;
                reinterpret_cast<u32x4 *>(o)[1] = b;
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i) o[i] = f[i];
            }
        } else {
            uint16_t h[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) h[i] = bf16_once(f[i], g);
            if constexpr (VEC) {
                u32x4 a;
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
                *reinterpret_cast<u32x4 *>(o) = a;
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i) o[i] = h[i];
            }
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
    const int upr = p.cols / kPer;
    const int64_t units = p.rows * upr;
    const bool vec = vector_rows(src, p.stride, p.rows, type == MOE_TYPE_F32 ? 4 : 2);
    const FastDiv by_upr(upr), by_global(p.globals ? p.rows_per_global : 1);
#define MOE_QUANT(F, V, S)                                                                                \
    hipLaunchKernelGGL((quantize_kernel<F, V, S>), dim3(grid_for(units)), dim3(kThreads), 0, s,          \
                       static_cast<const S *>(src), p.stride, units, upr, by_upr, p.globals, by_global, \
                       codes, scales)
#define MOE_QUANT_V(F, S)       \
    if (vec)                    \
        MOE_QUANT(F, true, S);  \
    else                        \
        MOE_QUANT(F, false, S);
    if (fmt == MOE_FMT_MXFP4 && type == MOE_TYPE_F32) {
        MOE_QUANT_V(MOE_FMT_MXFP4, float)
    } else if (fmt == MOE_FMT_MXFP4) {
        MOE_QUANT_V(MOE_FMT_MXFP4, uint16_t)
    } else if (type == MOE_TYPE_F32) {
        MOE_QUANT_V(MOE_FMT_E2M1, float)
    } else {
        MOE_QUANT_V(MOE_FMT_E2M1, uint16_t)
    }
#undef MOE_QUANT_V
#undef MOE_QUANT
    return hipGetLastError();
}

hipError_t launch_dequantize(int fmt, int type, const RowsParams &p, const uint8_t *codes,
                             const uint8_t *scales, void *dst, hipStream_t s) {
    if (p.rows == 0) return hipSuccess;
    const int upr = p.cols / kPer;
    const int64_t units = p.rows * upr;
    const bool vec = vector_rows(dst, p.stride, p.rows, type == MOE_TYPE_F32 ? 4 : 2);
    const FastDiv by_upr(upr), by_global(p.globals ? p.rows_per_global : 1);
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
