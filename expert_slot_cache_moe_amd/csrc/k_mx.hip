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

// Four consecutive outputs col .. col + 3 of a row of cols; `whole`: rows
// start on whole vectors of four and cols is a multiple of 4.
__device__ __forceinline__ void store4(float *o, int col, int cols, bool whole, f32x4 v) {
    if (whole) {
        if (col < cols) *reinterpret_cast<f32x4 *>(o + col) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < cols) o[col + e] = v[e];
    }
}
__device__ __forceinline__ void store4(uint16_t *o, int col, int cols, bool whole, f32x4 v) {
    if (whole) {
        if (col < cols)
            *reinterpret_cast<uint2 *>(o + col) =
                uint2{f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16),
                      f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16)};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < cols) o[col + e] = f32_to_bf16(v[e]);
    }
}

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

// Long runs: a block takes 256 rows of the matrix (with SwiGLU 128 gate and
// 128 up rows) and BT routes; each of its four waves multiplies a half of
// the rows with a half of the routes in 32 x 32 x 64 instructions, so an
// operand byte read from LDS meets 128 or BT / 2 rows of the other.  k
// passes in stages of 256 elements through two LDS buffers; the next
// stage's bytes wait in registers while this one is multiplied, and are
// written to the other buffer before the stage's last quarter is, so the
// matrix cores run on.
//
// In the 32 x 32 x 64 instruction lane l = 32 h + c holds, of row c, the 32
// elements of one scale block: half h takes blocks 4 h .. 4 h + 3 of a
// stage in four steps (on both operands alike), so that its four scale
// bytes are one dword, a byte of which the instruction selects.  The result
// lane holds rows 8 (i / 4) + 4 h + i % 4, i = 0..15, of column (route) c.
//
// An LDS row is the stage's 128 bytes of one operand row, eight 16-byte
// chunks (one MX block each); chunk j lies in slot j ^ (row & 7), which
// spreads the rows of an operand read over all banks.
constexpr int kTileRows = 256, kStageBlocks = 8, kStageBytes = 16 * kStageBlocks;
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Scale bytes of blocks b0 .. b0 + 7 of a row as two dwords; past the row's
// last block 0.  ALIGNED: rows are whole dwords.
template <bool ALIGNED>
__device__ __forceinline__ uint2 load_scales(const uint8_t *row, int b0, int nblk) {
    uint32_t v[2];
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const int b = b0 + 4 * d;
        if constexpr (ALIGNED) {
            const uint32_t t = *reinterpret_cast<const uint32_t *>(row + min(b, nblk - 4));
            v[d] = b < nblk ? t : 0u;
        } else {
            v[d] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t t = row[min(b + i, nblk - 1)];
                v[d] |= b + i < nblk ? t << (8 * i) : 0u;
            }
        }
    }
    return uint2{v[0], v[1]};
}

template <int BT, bool SWIGLU, bool ALIGNED, typename OUT>
__global__ __launch_bounds__(kThreads, 1) void mx_tile_kernel(MxParams p, const uint8_t *__restrict__ xc,
                                                              const uint8_t *__restrict__ xs,
                                                              const int32_t *__restrict__ n_runs,
                                                              const Run *__restrict__ runs,
                                                              const int32_t *__restrict__ routes, int R,
                                                              int row_tiles, OUT *__restrict__ out) {
    constexpr int kN = 4, kT = BT / 64;              // 32-row and 32-route tiles of a wave
    constexpr int kWLoads = kTileRows / 32, kXLoads = BT / 32;
    __shared__ __align__(16) uint8_t wbuf[2][kTileRows * kStageBytes];
    __shared__ __align__(16) uint8_t xbuf[2][BT * kStageBytes];
    __shared__ __align__(16) uint8_t wsc[2][kTileRows * kStageBlocks];
    __shared__ __align__(16) uint8_t xsc[2][kTileRows * kStageBlocks];   // a row for every thread

    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int c = lane & 31, h = lane / 32;
    // Consecutive workgroups go to the eight XCDs in turn; each XCD takes a
    // contiguous part of (run, row tile), so its L2 sees the runs of one
    // matrix and the row tiles of one run together.
    const int total = (n_runs != nullptr ? n_runs[0] : (R + BT - 1) / BT) * row_tiles;
    const int per = (total + 7) / 8;
    const int item = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
    if ((int)(blockIdx.x / 8) >= per || item >= total) return;
    const int ri = item / row_tiles, tile = item - ri * row_tiles;
    Run run;
    if (n_runs != nullptr)
        run = runs[ri];
    else
        run = Run{0, ri * BT, min(BT, R - ri * BT), 0};

    const int cols = SWIGLU ? p.n / 2 : p.n;
    constexpr int kCols = SWIGLU ? kTileRows / 2 : kTileRows;   // output columns of the block
    const int j0 = tile * kCols;
    const int nblk = p.k / 32, stages = (nblk + kStageBlocks - 1) / kStageBlocks;
    const int64_t row_bytes = (int64_t)nblk * 16;
    // LDS row r of the weights: with SwiGLU 64 gate rows, then their 64 up
    // rows, for each half of the block
    auto matrix_row = [&](int r) -> int64_t {
        if constexpr (SWIGLU) {
            const int j = min(j0 + (r >> 7) * 64 + (r & 63), cols - 1);
            return (int64_t)run.row * p.n + ((r & 64) ? cols : 0) + j;
        } else {
            return (int64_t)run.row * p.n + min(j0 + r, cols - 1);
        }
    };
    auto route_at = [&](int i) {
        const int at = run.start + min(i, run.count - 1);
        return n_runs != nullptr ? routes[at] : at;
    };

    const int wn = wave & 1, wt = wave >> 1;         // the wave's half of the rows, of the routes
    f32x16 acc[kN][kT];
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < kT; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

    if (run.row >= 0) {
        const uint8_t *wp[kWLoads], *xp[kXLoads];
        const int lr = tid / 8, chunk = (tid & 7) ^ (lr & 7);
#pragma unroll
        for (int i = 0; i < kWLoads; ++i) wp[i] = p.codes + matrix_row(32 * i + lr) * row_bytes;
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) xp[i] = xc + (int64_t)(route_at(32 * i + lr) / p.K) * row_bytes;
        const uint8_t *wsp = p.scales + matrix_row(tid) * nblk;
        const uint8_t *xsp = xs + (int64_t)(route_at(min(tid, BT - 1)) / p.K) * nblk;

        u32x4 wr[kWLoads], xr[kXLoads];
        uint2 wsr, xsr;
        auto fetch = [&](int st) {
            const int off = min(st * kStageBlocks + chunk, nblk - 1) * 16;
#pragma unroll
            for (int i = 0; i < kWLoads; ++i) wr[i] = *reinterpret_cast<const u32x4 *>(wp[i] + off);
#pragma unroll
            for (int i = 0; i < kXLoads; ++i) xr[i] = *reinterpret_cast<const u32x4 *>(xp[i] + off);
            wsr = load_scales<ALIGNED>(wsp, st * kStageBlocks, nblk);
            xsr = load_scales<ALIGNED>(xsp, st * kStageBlocks, nblk);
        };
        auto put = [&](int b) {
#pragma unroll
            for (int i = 0; i < kWLoads; ++i) *reinterpret_cast<u32x4 *>(&wbuf[b][i * 4096 + tid * 16]) = wr[i];
#pragma unroll
            for (int i = 0; i < kXLoads; ++i) *reinterpret_cast<u32x4 *>(&xbuf[b][i * 4096 + tid * 16]) = xr[i];
            *reinterpret_cast<uint2 *>(&wsc[b][tid * kStageBlocks]) = wsr;
            *reinterpret_cast<uint2 *>(&xsc[b][tid * kStageBlocks]) = xsr;
        };
        const int r0 = wn * 128 + c, t0 = wt * (BT / 2) + c;

        fetch(0);
        put(0);
        __syncthreads();
        for (int st = 0; st < stages; ++st) {
            const int b = st & 1;
            fetch(min(st + 1, stages - 1));
            uint32_t sa[kN], sb[kT];
#pragma unroll
            for (int i = 0; i < kN; ++i)
                sa[i] = *reinterpret_cast<const uint32_t *>(&wsc[b][(r0 + 32 * i) * kStageBlocks + 4 * h]);
#pragma unroll
            for (int i = 0; i < kT; ++i)
                sb[i] = *reinterpret_cast<const uint32_t *>(&xsc[b][(t0 + 32 * i) * kStageBlocks + 4 * h]);
#define MOE_READ(S)                                                                                       \
    u32x4 wa##S[kN], xb##S[kT];                                                                           \
    {                                                                                                     \
        const int slot = ((4 * h + S) ^ (c & 7)) * 16;                                                    \
        _Pragma("unroll") for (int i = 0; i < kT; ++i) xb##S[i] =                                         \
            *reinterpret_cast<const u32x4 *>(&xbuf[b][(t0 + 32 * i) * kStageBytes + slot]);               \
        _Pragma("unroll") for (int i = 0; i < kN; ++i) wa##S[i] =                                         \
            *reinterpret_cast<const u32x4 *>(&wbuf[b][(r0 + 32 * i) * kStageBytes + slot]);               \
    }
#define MOE_MULTIPLY(S)                                                                                   \
    _Pragma("unroll") for (int i = 0; i < kN; ++i) _Pragma("unroll") for (int j = 0; j < kT; ++j)         \
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(                                      \
            widen(wa##S[i]), widen(xb##S[j]), acc[i][j], kFp4, kFp4, S, (int)sa[i], S, (int)sb[j]);
            MOE_READ(0)
            MOE_READ(1)
            MOE_MULTIPLY(0)
            MOE_READ(2)
            MOE_MULTIPLY(1)
            MOE_READ(3)
            MOE_MULTIPLY(2)
            __builtin_amdgcn_sched_barrier(0);
            put(b ^ 1);   // read by nobody since the last barrier
            __builtin_amdgcn_sched_barrier(0);
            MOE_MULTIPLY(3)
#undef MOE_READ
#undef MOE_MULTIPLY
            __syncthreads();
        }
    }

    // lane (c, h) holds rows 8 g + 4 h .. + 3 (g = 0..3) of its row tiles for route c
    const bool whole = cols % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (4 * sizeof(OUT) - 1)) == 0;
#pragma unroll
    for (int j = 0; j < kT; ++j) {
        const int at = wt * (BT / 2) + 32 * j + c;
        if (at >= run.count) continue;
        OUT *o = out + (int64_t)route_at(at) * cols;
#pragma unroll
        for (int i = 0; i < (SWIGLU ? kN / 2 : kN); ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int col = j0 + wn * (kCols / 2) + 32 * i + 8 * g + 4 * h;
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = acc[i][j][4 * g + e];
                    if constexpr (SWIGLU) v[e] = silu(v[e]) * acc[i + kN / 2][j][4 * g + e];
                }
                store4(o, col, cols, whole, v);
            }
    }
}

}  // namespace

size_t mx_workspace_bytes(int P, int n, int k, int T, int K) {
    (void)n;
    return mx_ws(P, k, T, K).total;
}

namespace {

template <typename OUT>
hipError_t launch_stream(const MxParams &p, const uint8_t *xc, const uint8_t *xs, const int32_t *n_runs,
                         const Run *runs, const int32_t *routes, int R, int64_t max_runs, hipStream_t s) {
    const int cols = p.swiglu ? p.n / 2 : p.n;
    const dim3 grid((cols + kTile - 1) / kTile, (unsigned)max_runs);
    if (p.swiglu)
        hipLaunchKernelGGL((mx_stream_kernel<true, OUT>), grid, dim3(kThreads), 0, s, p, xc, xs, n_runs, runs,
                           routes, R, static_cast<OUT *>(p.out));
    else
        hipLaunchKernelGGL((mx_stream_kernel<false, OUT>), grid, dim3(kThreads), 0, s, p, xc, xs, n_runs, runs,
                           routes, R, static_cast<OUT *>(p.out));
    return hipGetLastError();
}

template <int BT, typename OUT>
hipError_t launch_tile(const MxParams &p, const uint8_t *xc, const uint8_t *xs, const int32_t *n_runs,
                       const Run *runs, const int32_t *routes, int R, int64_t max_runs, hipStream_t s) {
    const int per = p.swiglu ? kTileRows / 2 : kTileRows, cols = p.swiglu ? p.n / 2 : p.n;
    const int row_tiles = (cols + per - 1) / per;
    const unsigned grid = (unsigned)((max_runs * row_tiles + 7) / 8 * 8);
    const bool aligned = p.k % 128 == 0 && reinterpret_cast<uintptr_t>(p.scales) % 4 == 0;
#define MOE_TILE(S, A)                                                                                          \
    hipLaunchKernelGGL((mx_tile_kernel<BT, S, A, OUT>), dim3(grid), dim3(kThreads), 0, s, p, xc, xs, n_runs, runs, \
                       routes, R, row_tiles, static_cast<OUT *>(p.out))
    if (p.swiglu && aligned)
        MOE_TILE(true, true);
    else if (p.swiglu)
        MOE_TILE(true, false);
    else if (aligned)
        MOE_TILE(false, true);
    else
        MOE_TILE(false, false);
#undef MOE_TILE
    return hipGetLastError();
}

// Routes a run may hold, by the mean number of routes to a row: the widest
// tile that those fill.
int run_length_for(int R, int P, bool lists) {
    const int mean = lists ? R / std::min(R, P) : R;
    return mean >= 160 ? 256 : mean >= 64 ? 128 : mean >= 24 ? 64 : kRunLength;
}

template <typename OUT>
hipError_t launch_typed(const MxParams &p, const uint8_t *xc, const uint8_t *xs, const int32_t *n_runs,
                        const Run *runs, const int32_t *routes, int R, int run_length, int64_t max_runs,
                        hipStream_t s) {
    switch (run_length) {
    case 256: return launch_tile<256, OUT>(p, xc, xs, n_runs, runs, routes, R, max_runs, s);
    case 128: return launch_tile<128, OUT>(p, xc, xs, n_runs, runs, routes, R, max_runs, s);
    case 64: return launch_tile<64, OUT>(p, xc, xs, n_runs, runs, routes, R, max_runs, s);
    default: return launch_stream<OUT>(p, xc, xs, n_runs, runs, routes, R, max_runs, s);
    }
}

}  // namespace

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
    const int run_length = run_length_for(R, p.P, p.idx != nullptr);
    int64_t max_runs = (R + run_length - 1) / run_length;
    if (p.idx != nullptr) {
        max_runs = std::min<int64_t>(R, (int64_t)p.P + 1) + R / run_length;
        if (!reuse_lists) {
            const size_t lds = (2 * kGroupWaves + (size_t)p.P + 1) * 4;
            if (lds > 65536) {
                e = hipFuncSetAttribute(reinterpret_cast<const void *>(&mx_group_kernel),
                                        hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
                if (e != hipSuccess) return e;
            }
            hipLaunchKernelGGL(mx_group_kernel, dim3(1), dim3(kGroupThreads), lds, s, p.idx, R, p.P, run_length,
                               n_runs, runs, routes);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    } else {
        n_runs = nullptr;
    }
    return p.out_type == MOE_TYPE_F32
               ? launch_typed<float>(p, xc, xs, n_runs, runs, routes, R, run_length, max_runs, s)
               : launch_typed<uint16_t>(p, xc, xs, n_runs, runs, routes, R, run_length, max_runs, s);
}

}  // namespace moe
