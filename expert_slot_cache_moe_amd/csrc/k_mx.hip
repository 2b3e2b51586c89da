// MXFP4 x MXFP4 products over pool rows, on gfx950's scaled matrix
// instructions (v_mfma_scale_f32_16x16x128_f8f6f4 with both operands in
// 4-bit E2M1).
//
//   y[r] = W[idx[r]] q(x[r / K]),  W [n][k] and q(x) in MXFP4,
// optionally followed by silu(gate) * up over the two halves of y.
//
// The product of two E2M1 values and two powers of two is exact, so the
// only roundings are those of the fp32 sums.
//
// Operand layout: lane l = 16 q + c of a wave holds, of row c (A: matrix
// row, B: token), the 32 elements of scale block q of the 128-element step:
// 16 bytes of codes and one E8M0 byte, exactly one MX block.  The result
// lane holds rows 4 q .. 4 q + 3 of column (token) c.
//
// Steps past k: codes are read from the row's last block and both scale
// bytes are 0 (2^-127), so what they add is below 2^-240 and rounds to
// nothing in any sum (fp32 reaches down to 2^-149).
#include <algorithm>

#include "moe_internal.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kTile = 16;
constexpr int kStep = 128;                 // elements of one matrix instruction
constexpr int kFp4 = 4;                    // operand format code of E2M1

__device__ __forceinline__ i32x8 widen(u32x4 v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}
__device__ __forceinline__ f32x4 mfma(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(a), widen(b), c, kFp4, kFp4, 0, (int)sa, 0,
                                                            (int)sb);
}

__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t *p, float v) { *p = f32_to_bf16(v); }

// A run of routes that share a matrix row; row -1: routes without one.
struct Run {
    int32_t row, start, count, pad;
};

// Workspace: run count, runs, route ids sorted by row, quantised x.
struct MxWs {
    size_t n_runs, runs, routes, codes, scales, total;
    int64_t max_runs;
};
constexpr int kRunLength = kTile;

MxWs mx_ws(int P, int k, int T, int K) {
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    const int64_t R = (int64_t)T * K;
    MxWs w;
    w.max_runs = std::min<int64_t>(R, (int64_t)P + 1) + R / kRunLength;
    size_t off = 0;
    w.n_runs = off;
    off += up(4);
    w.runs = off;
    off += up((size_t)w.max_runs * sizeof(Run));
    w.routes = off;
    off += up((size_t)R * 4);
    w.codes = off;
    off += up((size_t)T * (k / 2));
    w.scales = off;
    off += up((size_t)T * (k / 32));
    w.total = off;
    return w;
}

// ------------------------------------------------------------------ grouping

// Routes sorted by matrix row with a counting sort in LDS (counts by
// atomics, one prefix sum over the rows), and each row's list cut into runs
// of at most run_length routes.  Routes without a row sort behind the last
// row, as runs of row -1.  The order inside a list is not fixed; every
// route's result is independent of its place.
constexpr int kGroupThreads = 1024, kGroupWaves = kGroupThreads / kWave;

__global__ __launch_bounds__(kGroupThreads) void mx_group_kernel(const int32_t *__restrict__ idx, int R, int P,
                                                                 int run_length, int32_t *__restrict__ n_runs,
                                                                 Run *__restrict__ runs,
                                                                 int32_t *__restrict__ routes) {
    extern __shared__ __align__(16) int32_t lds[];
    int32_t *wsum = lds;         // [2][kGroupWaves]
    int32_t *cnt = lds + 2 * kGroupWaves;   // [P + 1]
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    for (int r = tid; r <= P; r += kGroupThreads) cnt[r] = 0;
    __syncthreads();
    for (int i = tid; i < R; i += kGroupThreads) {
        const int r = idx[i];
        atomicAdd(&cnt[r >= 0 && r < P ? r : P], 1);
    }
    __syncthreads();
    const int per = (P + kGroupThreads) / kGroupThreads;   // rows 0..P
    const int r0 = tid * per;
    int n = 0, t = 0;
    for (int i = 0; i < per; ++i)
        if (r0 + i <= P) {
            const int v = cnt[r0 + i];
            n += v;
            t += (v + run_length - 1) / run_length;
        }
    const int n_in = wave_inclusive_sum(n), t_in = wave_inclusive_sum(t);
    if (lane == kWave - 1) {
        wsum[wave] = n_in;
        wsum[kGroupWaves + wave] = t_in;
    }
    __syncthreads();
    int start = n_in - n, run = t_in - t, total = 0;
    for (int v = 0; v < kGroupWaves; ++v) {
        start += v < wave ? wsum[v] : 0;
        run += v < wave ? wsum[kGroupWaves + v] : 0;
        total += wsum[kGroupWaves + v];
    }
    for (int i = 0; i < per; ++i)
        if (r0 + i <= P) {
            const int v = cnt[r0 + i];
            cnt[r0 + i] = start;
            for (int o = 0; o < v; o += run_length)
                runs[run++] = Run{r0 + i < P ? r0 + i : -1, start + o, min(run_length, v - o), 0};
            start += v;
        }
    if (tid == 0) n_runs[0] = total;
    __syncthreads();
    for (int i = tid; i < R; i += kGroupThreads) {
        const int r = idx[i];
        routes[atomicAdd(&cnt[r >= 0 && r < P ? r : P], 1)] = i;
    }
}

// ------------------------------------------------------------------ product

constexpr int kWaves = 4, kThreads = kWaves * kWave;

// One block: 16 output columns (with SwiGLU 16 gate and 16 up rows of the
// matrix) for one run of up to 16 routes; the waves take every fourth step
// of k and add their sums in LDS, in wave order.
template <bool SWIGLU, typename OUT>
__global__ __launch_bounds__(kThreads) void mx_stream_kernel(MxParams p, const uint8_t *__restrict__ xc,
                                                             const uint8_t *__restrict__ xs,
                                                             const int32_t *__restrict__ n_runs,
                                                             const Run *__restrict__ runs,
                                                             const int32_t *__restrict__ routes, int R,
                                                             OUT *__restrict__ out) {
    constexpr int kM = SWIGLU ? 2 : 1;
    __shared__ f32x4 part[kWaves][kM][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int c = lane & (kTile - 1), q = lane / kTile;
    Run run;
    if (n_runs != nullptr) {
        if ((int)blockIdx.y >= n_runs[0]) return;
        run = runs[blockIdx.y];
    } else {
        run = Run{0, (int)blockIdx.y * kRunLength, min(kRunLength, R - (int)blockIdx.y * kRunLength), 0};
    }
    const int cols = SWIGLU ? p.n / 2 : p.n;
    const int j0 = blockIdx.x * kTile;
    const int at = run.start + min(c, run.count - 1);
    const int route = n_runs != nullptr ? routes[at] : at;
    f32x4 acc[kM];
#pragma unroll
    for (int m = 0; m < kM; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (run.row >= 0) {
        const int nblk = p.k / 32, steps = (p.k + kStep - 1) / kStep;
        const int64_t token = route / p.K;
        const uint8_t *bx = xc + token * (p.k / 2), *bs = xs + token * nblk;
        const uint8_t *ax[kM], *as[kM];
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            const int64_t r = (int64_t)run.row * p.n + m * cols + min(j0 + c, cols - 1);
            ax[m] = p.codes + r * (p.k / 2);
            as[m] = p.scales + r * nblk;
        }
        for (int s = wave; s < steps; s += kWaves) {
            const int b = 4 * s + q, bc = min(b, nblk - 1);
            const u32x4 bv = reinterpret_cast<const u32x4 *>(bx)[bc];
            const uint32_t sb = b < nblk ? bs[bc] : 0u;
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                const u32x4 av = reinterpret_cast<const u32x4 *>(ax[m])[bc];
                const uint32_t sa = b < nblk ? as[m][bc] : 0u;
                acc[m] = mfma(av, sa, bv, sb, acc[m]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < kM; ++m) part[wave][m][lane] = acc[m];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int m = 0; m < kM; ++m)
        for (int v = 1; v < kWaves; ++v) acc[m] += part[v][m][lane];
    if (c >= run.count) return;
    OUT *o = out + (int64_t)route * cols + j0 + 4 * q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (j0 + 4 * q + i < cols) store_out(o + i, SWIGLU ? silu(acc[0][i]) * acc[kM - 1][i] : acc[0][i]);
}

}  // namespace

size_t mx_workspace_bytes(int P, int n, int k, int T, int K) {
    (void)n;
    return mx_ws(P, k, T, K).total;
}

hipError_t launch_mx_product(const MxParams &p, bool reuse_lists, hipStream_t s) {
    const int R = p.T * p.K;
    if (R == 0) return hipSuccess;
    const MxWs L = mx_ws(p.P, p.k, p.T, p.K);
    int32_t *n_runs = reinterpret_cast<int32_t *>(p.ws + L.n_runs);
    Run *runs = reinterpret_cast<Run *>(p.ws + L.runs);
    int32_t *routes = reinterpret_cast<int32_t *>(p.ws + L.routes);
    uint8_t *xc = p.ws + L.codes, *xs = p.ws + L.scales;
    RowsParams rp{};
    rp.rows = p.T;
    rp.cols = p.k;
    rp.stride = p.x_stride;
    hipError_t e = launch_quantize(MOE_FMT_MXFP4, MOE_TYPE_BF16, rp, p.x, xc, xs, s);
    if (e != hipSuccess) return e;
    int64_t n_items = (R + kRunLength - 1) / kRunLength;
    if (p.idx != nullptr) {
        n_items = L.max_runs;
        if (!reuse_lists) {
            const size_t lds = (2 * kGroupWaves + (size_t)p.P + 1) * 4;
            if (lds > 65536) {
                e = hipFuncSetAttribute(reinterpret_cast<const void *>(&mx_group_kernel),
                                        hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
                if (e != hipSuccess) return e;
            }
            hipLaunchKernelGGL(mx_group_kernel, dim3(1), dim3(kGroupThreads), lds, s, p.idx, R, p.P, kRunLength,
                               n_runs, runs, routes);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    } else {
        n_runs = nullptr;
    }
    const int cols = p.swiglu ? p.n / 2 : p.n;
    const dim3 grid((cols + kTile - 1) / kTile, (unsigned)n_items);
#define MOE_MX(S, O)                                                                                         \
    hipLaunchKernelGGL((mx_stream_kernel<S, O>), grid, dim3(kThreads), 0, s, p, xc, xs, n_runs, runs, routes, \
                       R, static_cast<O *>(p.out))
    if (p.swiglu && p.out_type == MOE_TYPE_F32)
        MOE_MX(true, float);
    else if (p.swiglu)
        MOE_MX(true, uint16_t);
    else if (p.out_type == MOE_TYPE_F32)
        MOE_MX(false, float);
    else
        MOE_MX(false, uint16_t);
#undef MOE_MX
    return hipGetLastError();
}

}  // namespace moe
