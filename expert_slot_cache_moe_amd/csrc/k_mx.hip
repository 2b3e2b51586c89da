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
#include <type_traits>

#include "k_rows.inc"

namespace moe {
namespace {

using namespace rows_detail;

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

// Two fp32 rounded to bf16, by the hardware's conversion (to nearest, ties to even).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

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
            *reinterpret_cast<uint2 *>(o + col) = uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
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
constexpr int kRunLength = kTile;   // the shortest run

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
constexpr int kGroupThreads = 1024, kGroupWaves = kGroupThreads / kWave, kGroupAhead = 8;
// LDS of the list-making block: counters of up to 32769 rows (131 KB), or
// fewer and the sorted ids.
constexpr int kPrepareLds = 144 << 10;

// The next free place of `row`, one for each active lane.  Lanes that share
// the first lane's row take theirs with one addition (one matrix for all
// routes is a usual case, and 64 additions to one word take 64 turns).
__device__ __forceinline__ int place(int32_t *cnt, int row) {
    const int first = __builtin_amdgcn_readfirstlane(row);
    const uint64_t same = __ballot(row == first);
    if (row != first) return atomicAdd(&cnt[row], 1);
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0u));
    int base = 0;
    if (before == 0) base = atomicAdd(&cnt[row], __popcll(same));
    return __builtin_amdgcn_readfirstlane(base) + before;
}

// Block 0 makes the lists; the others, if any, quantise x, so the one goes on
// beside the other.  lists = 0: every block quantises.  staged: the sorted
// ids are put together in LDS and written in order (a scattered store of 64
// lanes takes 64 turns: 24576 ids 24 -> 12 us), where they fit: up to some
// 36000.  One block makes all lists, so their time grows with the ids and
// steps up there (a product over 256 matrices of 256 x 256, a call: 32768
// ids 32 us, 36000 36, 37600 47, 65536 72, 131072 131).
struct PrepareParams {
    const int32_t *idx;
    int32_t R, P, run_length, lists, staged;
    int32_t *n_runs;
    Run *runs;
    int32_t *routes;
    const uint16_t *x;
    int64_t x_stride, units;             // of 8 elements
    int32_t upr;
    FastDiv by_upr;
    uint8_t *codes, *scales;
};

template <bool VEC>
__global__ __launch_bounds__(kGroupThreads) void mx_prepare_kernel(PrepareParams a) {
    extern __shared__ __align__(16) int32_t lds[];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    if ((int)blockIdx.x >= a.lists) {
        const int64_t step = (int64_t)(gridDim.x - a.lists) * kGroupThreads;
        for (int64_t u = (int64_t)(blockIdx.x - a.lists) * kGroupThreads + tid; u < a.units; u += step) {
            const int64_t row = (int64_t)a.by_upr((uint64_t)u);
            float f[kPer];
            load8<VEC>(a.x + row * a.x_stride + (u - row * a.upr) * kPer, f);
            uint32_t sc;
            const uint32_t c = mx_codes(f, quad_max(amax_bits(f)), sc);
            reinterpret_cast<uint32_t *>(a.codes)[u] = c;
            if ((tid & 3) == 0) a.scales[u / 4] = (uint8_t)sc;
        }
        return;
    }
    const int R = a.R, P = a.P, run_length = a.run_length;
    int32_t *wsum = lds;                    // [2][kGroupWaves]
    int32_t *cnt = lds + 2 * kGroupWaves;   // [P + 1]
    int32_t *sorted = cnt + P + 1;          // [R], staged
    for (int r = tid; r <= P; r += kGroupThreads) cnt[r] = 0;
    __syncthreads();
    // eight ids of a thread at a time are on their way together
    auto each = [&](auto visit) {
        for (int i0 = tid; i0 < R; i0 += kGroupAhead * kGroupThreads) {
            int r[kGroupAhead];
#pragma unroll
            for (int k = 0; k < kGroupAhead; ++k) r[k] = a.idx[min(i0 + k * kGroupThreads, R - 1)];
#pragma unroll
            for (int k = 0; k < kGroupAhead; ++k)
                if (i0 + k * kGroupThreads < R)
                    visit(i0 + k * kGroupThreads, r[k] >= 0 && r[k] < P ? r[k] : P);
        }
    };
    each([&](int, int row) { place(cnt, row); });
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
                a.runs[run++] = Run{r0 + i < P ? r0 + i : -1, start + o, min(run_length, v - o), 0};
            start += v;
        }
    if (tid == 0) a.n_runs[0] = total;
    __syncthreads();
    if (a.staged) {
        each([&](int i, int row) { sorted[place(cnt, row)] = i; });
        __syncthreads();
        for (int i = tid; i < R; i += kGroupThreads) a.routes[i] = sorted[i];
    } else {
        each([&](int i, int row) { a.routes[place(cnt, row)] = i; });
    }
}

// ------------------------------------------------------------------ product

constexpr int kWaves = 4, kThreads = kWaves * kWave;

// Short runs: 16 routes of one matrix row at a time against columns of
// 16, the matrix straight from memory to registers (it is read once, so
// nothing is gained by passing it through LDS), x quantised where it is
// needed, so that no launch of its own has to do that first.
//
// Lists of routes come in three ways:
//   kRuns    from mx_prepare_kernel (or, without ids, consecutive rows);
//   kByRoute slot r is route r: the first route of its matrix row takes all
//            of that row's routes, the others leave;
//   kByRow   slot i is matrix row i, slot P the routes without a row.
// The last two look through idx in the block itself: no launch for the lists,
// but every block reads all ids.  1200 routes over 160 matrices 15.7 us, from
// prepared lists 19.7; 2000 over 256 77.9 and 75.9: up to 2048.
enum ListMode : int { kRuns, kByRoute, kByRow };
constexpr int kInlineRoutes = 2048, kIdxPerThread = kInlineRoutes / kThreads;
static_assert(kIdxPerThread * kWaves <= kWave, "one lane for each count");

// A barrier that orders LDS alone: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

struct ListLds {
    int32_t routes[kInlineRoutes];
    int32_t counts[kIdxPerThread * kWaves];
};

struct RouteList {
    int row = -1, count = 0, start = 0;
    const int32_t *at = nullptr;             // in LDS or memory; NULL: start, start + 1, ...
    __device__ __forceinline__ int route(int i) const { return at != nullptr ? at[i] : start + i; }
};

// The ids of idx that one of 256 threads looks through.
struct IdxPart {
    int32_t r[kIdxPerThread];
    // (no load here is conditional, so the compiler can count what is in flight)
    __device__ __forceinline__ void load(const int32_t *idx, int tid, int R) {
#pragma unroll
        for (int k = 0; k < kIdxPerThread; ++k) r[k] = idx[min(k * kThreads + tid, R - 1)];
    }
};

// The matrix row of an inline list's slot; -1: routes without a row.
__device__ __forceinline__ int slot_row(const MxParams &p, int mode, int slot) {
    const int row = mode == kByRoute ? p.idx[slot] : slot;
    return __builtin_amdgcn_readfirstlane(row < 0 || row >= p.P ? -1 : row);
}

// Collects the routes of `row`, ascending, into the block's list and returns
// their number.  (Blocks that share a list must agree on its order.)
__device__ __forceinline__ int collect(const IdxPart &part, ListLds &lds, const MxParams &p, int row, int R) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    uint64_t m[kIdxPerThread];
#pragma unroll
    for (int k = 0; k < kIdxPerThread; ++k) {
        const int v = part.r[k] < 0 || part.r[k] >= p.P ? -1 : part.r[k];
        m[k] = __ballot(k * kThreads + tid < R && v == row);
        if (lane == 0) lds.counts[k * kWaves + wave] = __popcll(m[k]);
    }
    lds_barrier();
    const int n = lane < kIdxPerThread * kWaves ? lds.counts[lane] : 0;
    const int incl = wave_inclusive_sum(n);
#pragma unroll
    for (int k = 0; k < kIdxPerThread; ++k) {
        if (m[k] == 0) continue;
        const int base = __builtin_amdgcn_readlane(incl - n, k * kWaves + wave);
        if ((m[k] >> lane) & 1)
            lds.routes[base + __builtin_amdgcn_mbcnt_hi((uint32_t)(m[k] >> 32),
                                                        __builtin_amdgcn_mbcnt_lo((uint32_t)m[k], 0u))] =
                k * kThreads + tid;
    }
    lds_barrier();
    return __builtin_amdgcn_readlane(incl, kWave - 1);
}

// The list of slot `slot` of a launch without inline lists; false: none.
__device__ __forceinline__ bool run_list(RouteList &l, int slot, int run_length, const int32_t *n_runs,
                                         const Run *runs, const int32_t *routes, int R) {
    if (n_runs != nullptr) {
        if (slot >= n_runs[0]) return false;
        const Run run = runs[slot];
        l.row = run.row;
        l.count = run.count;
        l.at = routes + run.start;
    } else {
        l.row = 0;
        l.start = slot * run_length;
        l.count = min(run_length, R - l.start);
    }
    return true;
}

// Zeros in columns [j0, j0 + width) of every route of a list, by THREADS
// threads, 16 bytes at a time where rows are whole vectors (j0 and the
// unclipped width always are).
template <int THREADS>
__device__ __forceinline__ void zero_rows(const MxParams &p, const RouteList &l, int cols, int j0, int width, int tid) {
    const int size = p.out_type == MOE_TYPE_F32 ? 4 : 2;
    const int64_t row_bytes = (int64_t)cols * size;
    const bool whole = row_bytes % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
    const int unit = whole ? 16 : size, units = min(width, cols - j0) * size / unit;
    if (units <= 0) return;
    uint8_t *out = static_cast<uint8_t *>(p.out) + (int64_t)j0 * size;
    for (int i = tid; i < l.count * units; i += THREADS) {
        const int t = i / units;
        uint8_t *o = out + l.route(t) * row_bytes + (int64_t)(i - t * units) * unit;
        if (whole)
            *reinterpret_cast<u32x4 *>(o) = u32x4{0u, 0u, 0u, 0u};
        else if (size == 4)
            *reinterpret_cast<uint32_t *>(o) = 0u;
        else
            *reinterpret_cast<uint16_t *>(o) = 0;
    }
}

// Four columns of a route's result: the sums, or silu(gate) * up of them.
template <bool SWIGLU, int kM>
__device__ __forceinline__ void store_columns(const MxParams &p, bool f32_out, int route, int cols, int col,
                                              bool whole, f32x4 (&v)[kM]) {
    if constexpr (SWIGLU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[0][i] = silu(v[0][i]) * v[kM - 1][i];
    }
    if (f32_out)
        store4(static_cast<float *>(p.out) + (int64_t)route * cols, col, cols, whole, v[0]);
    else
        store4(static_cast<uint16_t *>(p.out) + (int64_t)route * cols, col, cols, whole, v[0]);
}

// The scale bytes of a row for U steps: lane quarter q uses byte q of each
// step's four.  VEC: whole, aligned vectors (k a multiple of 128 U).
template <int U, bool VEC> struct StepScales {
    uint32_t v[U];
    __device__ __forceinline__ void load(const uint8_t *row, int s0, int nblk, int q) {
        if constexpr (VEC && U == 4) {
            const u32x4 t = *reinterpret_cast<const u32x4 *>(row + 4 * s0);
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = t[u];
        } else if constexpr (VEC && U == 2) {
            const uint2 t = *reinterpret_cast<const uint2 *>(row + 4 * s0);
            v[0] = t.x;
            v[1] = t.y;
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = 4 * (s0 + u) + q;
                const uint32_t t = row[min(b, nblk - 1)];
                v[u] = b < nblk ? t : 0u;
            }
        }
    }
    __device__ __forceinline__ uint32_t at(int u, int q) const { return VEC ? v[u] >> (8 * q) : v[u]; }
};

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// 32 bf16 as an MX block: codes and scale byte (0xFF and zeros where one of
// them is NaN or infinite).  x / scale is exact, so the scaled conversion's
// one rounding is the format's.
__device__ __forceinline__ u32x4 quantize_block(const u32x4 (&x)[4], uint32_t &scale) {
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int d = 0; d < 4; ++d)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x[i][d] & 0x7fff7fffu));
    const int a = max((int)m[0], (int)m[1]);
    const bool bad = a >= 0x7f80;
    const int e = max((a >> 7) - 2, 0);
    const float f = __uint_as_float((uint32_t)e << 23);
    u32x4 c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t t = 0;
        // (a bit cast of a vector's element itself would take its first one)
#define MOE_CVT(B)                                                                                    \
    {                                                                                                 \
        const uint32_t pair = x[i][B];                                                                \
        t = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(t, __builtin_bit_cast(bf16x2, pair), f, B);     \
    }
        MOE_CVT(0)
        MOE_CVT(1)
        MOE_CVT(2)
        MOE_CVT(3)
#undef MOE_CVT
        c[i] = bad ? 0u : t;
    }
    scale = bad ? 0xFFu : (uint32_t)e;
    return c;
}

// A 64-byte block of a row of x, as 32 bf16.
__device__ __forceinline__ void load_block(const uint16_t *x, bool vec, u32x4 (&v)[4]) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const u32x4 *>(x)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) v[i][d] = x[8 * i + 2 * d] | ((uint32_t)x[8 * i + 2 * d + 1] << 16);
    }
}

// A lane's codes and scales of U steps of kM matrix rows.
template <int U, bool VEC, int kM> struct MatrixChunk {
    u32x4 a[kM][U];
    StepScales<U, VEC> s[kM];
    __device__ __forceinline__ void load(const uint8_t *const (&ax)[kM], const uint8_t *const (&as)[kM], int s0,
                                         int nblk, int q) {
#pragma unroll
        for (int m = 0; m < kM; ++m) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = 4 * (s0 + u) + q;
                a[m][u] = reinterpret_cast<const u32x4 *>(ax[m])[VEC ? b : min(b, nblk - 1)];
            }
            s[m].load(as[m], s0, nblk, q);
        }
    }
};

// Few blocks: the four waves of a block share 16 output columns (with
// SwiGLU 16 gate and 16 up rows) and split k, every fourth chunk of U steps
// each; their sums are added in LDS, in wave order.  A lane's part of x for
// one step is one whole MX block of one token, quantised in registers.
//
// A token's 8 routes of 1024 x 2048 (9 MB) take 5.4 us: the latency of ids,
// matrix and sums one behind the other.
template <bool SWIGLU, int U, bool VEC, bool INLINE>
__global__ __launch_bounds__(kThreads) void mx_split_kernel(MxParams p, int mode, bool x_vec,
                                                            const int32_t *__restrict__ n_runs,
                                                            const Run *__restrict__ runs,
                                                            const int32_t *__restrict__ routes, int R) {
    constexpr int kM = SWIGLU ? 2 : 1;
    __shared__ f32x4 part[kWaves][kM][kWave];
    __shared__ ListLds lds;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int c = lane & (kTile - 1), q = lane / kTile;
    const int cols = SWIGLU ? p.n / 2 : p.n;
    const int j0 = blockIdx.x * kTile;
    const int nblk = p.k / 32, steps = (p.k + kStep - 1) / kStep;
    const int last = (steps - 1) / U * U;    // the last chunk; requests past it repeat it

    MatrixChunk<U, VEC, kM> w;
    const uint8_t *ax[kM], *as[kM];
    RouteList l;
    auto request = [&](int row) {
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            const int64_t r = (int64_t)max(row, 0) * p.n + m * cols + min(j0 + c, cols - 1);
            ax[m] = p.codes + r * nblk * 16;
            as[m] = p.scales + r * nblk;
        }
        w.load(ax, as, min(wave * U, last), nblk, q);
    };
    if constexpr (INLINE) {
        // the matrix is requested right behind the ids, before they are looked through
        IdxPart part;
        part.load(p.idx, tid, R);
        l.row = slot_row(p, mode, blockIdx.y);
        request(l.row);
        l.count = collect(part, lds, p, l.row, R);
        l.at = lds.routes;
        if (l.count == 0 || (mode == kByRoute && lds.routes[0] < (int)blockIdx.y)) return;
    } else {
        if (!run_list(l, blockIdx.y, kTile, n_runs, runs, routes, R)) return;
        request(l.row);
    }
    if (l.row < 0) {
        zero_rows<kThreads>(p, l, cols, j0, kTile, tid);
        return;
    }
    const bool f32_out = p.out_type == MOE_TYPE_F32;
    const bool whole = cols % 4 == 0 && (reinterpret_cast<uintptr_t>(p.out) & (f32_out ? 15 : 7)) == 0;

    for (int base = 0; base < l.count; base += kTile) {
        f32x4 acc[kM];
#pragma unroll
        for (int m = 0; m < kM; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int route = l.route(min(base + c, l.count - 1));
        const uint16_t *xr = p.x + (int64_t)(route / p.K) * p.x_stride;
        for (int s0 = wave * U; s0 < steps; s0 += kWaves * U) {
            // the first pass's first chunk is there already
            if (base > 0 || s0 != wave * U) w.load(ax, as, s0, nblk, q);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = 4 * (s0 + u) + q;
                u32x4 xv[4];
                load_block(xr + 32 * (VEC ? b : min(b, nblk - 1)), x_vec, xv);
                uint32_t sb;
                const u32x4 bv = quantize_block(xv, sb);
                if (!VEC && b >= nblk) sb = 0u;
#pragma unroll
                for (int m = 0; m < kM; ++m) acc[m] = mfma(w.a[m][u], w.s[m].at(u, q), bv, sb, acc[m]);
            }
        }
        if (base > 0) lds_barrier();         // the last pass has read its sums
#pragma unroll
        for (int m = 0; m < kM; ++m) part[wave][m][lane] = acc[m];
        lds_barrier();
        if (wave != 0 || base + c >= l.count) continue;
        f32x4 v[kM];
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            v[m] = part[0][m][lane];
#pragma unroll
            for (int o = 1; o < kWaves; ++o) v[m] += part[o][m][lane];
        }
        store_columns<SWIGLU>(p, f32_out, route, cols, j0 + 4 * q, whole, v);
    }
}

// Many blocks: each of the four waves has 16 output columns (with SwiGLU 16
// gate and 16 up rows; without, 32 columns) of its own over all of k, and
// the block quantises its routes' x into LDS once for all four, 64 MX
// blocks of k at a time.  LDS holds codes by (block of k, token), 16 bytes
// each, so that an operand read is 1 KB in a row.
//
// A wave's loads return in order.  So the first part of x is requested
// first and the matrix behind it: x is quantised while the matrix, two
// chunks of U steps at once, is on its way.  Where those are all of k they
// serve every pass over a long list.
//
// 1200 routes spread over 160 matrices of 512 x 1024 (45 MB) take 15 us, 3.0
// TB/s: bound by latency, as the blocks of a launch ask for their ids, their
// x and their matrix in turn.  Skewed lists (the longest of 50 routes) take
// 20: each further pass of a block adds 4.
//
// Three waves to a SIMD, though four would fit (three / four, us: 1200 routes
// over 160 matrices, k 1024 15.3 / 18.8; 80 over 64, k 2048 20.0 / 24.8; 600
// over 200, k 512 11.3 / 10.3).
constexpr int kSpanBlocks = 64;

template <bool SWIGLU, bool VEC, bool INLINE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(3, 3))) void mx_stream_kernel(
    MxParams p, int mode, bool x_vec, int slots, int pass_blocks, const int32_t *__restrict__ n_runs,
    const Run *__restrict__ runs, const int32_t *__restrict__ routes, int R) {
    constexpr int kM = 2, U = 2;
    constexpr int kCols = SWIGLU ? kTile : 2 * kTile;       // output columns of a wave
    __shared__ __align__(16) u32x4 xc[kSpanBlocks][kTile];
    __shared__ uint8_t xs[kSpanBlocks][kTile];
    __shared__ ListLds lds;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int c = lane & (kTile - 1), q = lane / kTile;
    // Lists vary fastest: workgroups go to the eight XCDs in turn, and blocks
    // with work and blocks without (no such list, no such pass) must not fall
    // to different ones.
    const int slot = blockIdx.x % slots, rest = blockIdx.x / slots;
    const int pass = rest % pass_blocks, cb = rest / pass_blocks;
    const int cols = SWIGLU ? p.n / 2 : p.n;
    const int j0 = (cb * kWaves + wave) * kCols;
    const int nblk = p.k / 32, steps = (p.k + kStep - 1) / kStep;
    const int last = (steps - 1) / U * U;    // the last chunk; requests past it repeat it

    RouteList l;
    if constexpr (INLINE) {
        IdxPart part;
        part.load(p.idx, tid, R);
        l.row = slot_row(p, mode, slot);
        l.count = collect(part, lds, p, l.row, R);
        l.at = lds.routes;
        if (l.count <= pass * kTile || (mode == kByRoute && lds.routes[0] < slot)) return;
    } else if (!run_list(l, slot, kTile, n_runs, runs, routes, R)) {
        return;
    }
    if (l.row < 0) {
        if (pass == 0) zero_rows<kThreads>(p, l, cols, cb * kWaves * kCols, kWaves * kCols, tid);
        return;
    }

    // x: lanes over blocks of one token, or of two or four where k is short
    const int shift = nblk > 32 ? 6 : nblk > 16 ? 5 : 4;
    const int xb = tid & ((1 << shift) - 1), xt = tid >> shift, per = kThreads >> shift;
    u32x4 xv[4];
    auto x_load = [&](int base, int b0, int t) {     // rows past the list and blocks past the row repeat the last
        const int64_t token = l.route(min(base + t, l.count - 1)) / p.K;
        load_block(p.x + token * p.x_stride + 32 * min(b0 + xb, nblk - 1), x_vec, xv);
    };
    auto x_put = [&](int t) {
        uint32_t sb;
        const u32x4 codes = quantize_block(xv, sb);
        xc[xb][t] = codes;
        xs[xb][t] = (uint8_t)sb;
    };
    x_load(pass * kTile, 0, xt);

    MatrixChunk<U, VEC, kM> w[2];
    const uint8_t *ax[kM], *as[kM];
#pragma unroll
    for (int m = 0; m < kM; ++m) {
        const int j = SWIGLU ? min(j0 + c, cols - 1) + m * cols : min(j0 + m * kTile + c, cols - 1);
        const int64_t r = (int64_t)l.row * p.n + j;
        ax[m] = p.codes + r * nblk * 16;
        as[m] = p.scales + r * nblk;
    }
    auto request = [&](MatrixChunk<U, VEC, kM> &to, int s0) { to.load(ax, as, s0, nblk, q); };
    request(w[0], 0);
    request(w[1], min(U, last));
    const bool f32_out = p.out_type == MOE_TYPE_F32;
    const bool whole = cols % 4 == 0 && (reinterpret_cast<uintptr_t>(p.out) & (f32_out ? 15 : 7)) == 0;

    bool again = false;
    for (int base = pass * kTile; base < l.count; base += pass_blocks * kTile) {
        f32x4 acc[kM];
#pragma unroll
        for (int m = 0; m < kM; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int live = min(l.count - base, kTile);
        if (again && steps > 2 * U) {
            request(w[0], 0);
            request(w[1], min(U, last));
        }
        for (int b0 = 0; b0 < nblk; b0 += kSpanBlocks) {
            const int nb = min(kSpanBlocks, nblk - b0);
            if (again) {
                lds_barrier();               // the span before has been read
                x_load(base, b0, xt);
            }
            again = true;
            x_put(xt);
            for (int t = xt + per; t < live; t += per) {
                x_load(base, b0, t);
                x_put(t);
            }
            lds_barrier();
            const int s_end = (min(b0 + kSpanBlocks, nblk) + 3) / 4;
            auto chunk = [&](int s0, const MatrixChunk<U, VEC, kM> &m0) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int b = 4 * (s0 + u) + q - b0, bc = VEC ? b : min(b, nb - 1);
                    const int tc = min(c, live - 1);
                    const u32x4 bv = xc[bc][tc];
                    const uint32_t sb = VEC || b < nb ? xs[bc][tc] : 0u;
#pragma unroll
                    for (int m = 0; m < kM; ++m) acc[m] = mfma(m0.a[m][u], m0.s[m].at(u, q), bv, sb, acc[m]);
                }
            };
            // Where the two chunks are not all of k, each is followed by the
            // request for the chunk after next: behind the products that free
            // its registers, and on no branch, or the compiler takes other
            // registers and waits for the requests to copy them.
            auto multiply = [&](auto whole_k) {
                for (int s0 = b0 / 4; s0 < s_end; s0 += 2 * U) {
                    chunk(s0, w[0]);
                    if constexpr (!decltype(whole_k)::value) {
                        __builtin_amdgcn_sched_barrier(0);
                        request(w[0], min(s0 + 2 * U, last));
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (s0 + U < s_end) chunk(s0 + U, w[1]);
                    if constexpr (!decltype(whole_k)::value) {
                        __builtin_amdgcn_sched_barrier(0);
                        request(w[1], min(s0 + 3 * U, last));
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            };
            if (steps > 2 * U)
                multiply(std::false_type{});
            else
                multiply(std::true_type{});
        }
        if (c < live) {
            const int route = l.route(base + c);
            if constexpr (SWIGLU) {
                f32x4 v[kM] = {acc[0], acc[1]};
                store_columns<true>(p, f32_out, route, cols, j0 + 4 * q, whole, v);
            } else {
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                    f32x4 v[1] = {acc[m]};
                    store_columns<false>(p, f32_out, route, cols, j0 + m * kTile + 4 * q, whole, v);
                }
            }
        }
    }
}

// Long runs: a block takes 256 or 128 rows of the matrix (with SwiGLU a half
// gate and a half up rows) and BT routes, in 32 x 32 x 64 instructions.  At BT 256 each
// of its four waves multiplies a half of the rows with a half of the routes,
// so an operand byte read from LDS meets 128 rows of the other.  At 128 and
// 64 each wave multiplies a quarter of the rows with all routes, and tiles
// of 32 routes that the run does not reach are left out: the instructions
// follow the run's length in steps of 32.
//
// k passes in stages of 256 elements through two LDS buffers.  The stage
// after the next (at BT 256, for want of registers, the next) is on its way
// to registers while one is multiplied; the next is written from registers
// to the other buffer before the stage's last quarter is multiplied, so the
// matrix cores run on.
//
// In the 32 x 32 x 64 instruction lane l = 32 h + c holds, of row c, the 32
// elements of one scale block: half h takes blocks 4 h .. 4 h + 3 of a
// stage in four steps (on both operands alike), so that its four scale
// bytes are one dword, a byte of which the instruction selects.  The result
// lane holds rows 8 (i / 4) + 4 h + i % 4, i = 0..15, of column (route) c.
//
// An LDS row is the stage's 128 bytes of one operand row, eight 16-byte
// chunks (one MX block each); chunk j lies in slot j ^ (row / 2 % 8): two rows
// fill the 64 banks, and the 16 rows that are read at once hit each bank once.
constexpr int kStageBlocks = 8, kStageBytes = 16 * kStageBlocks;
// Rows of the matrix a block takes: at BT 256 as many as the registers hold;
// below, where the matrix's bytes bound the kernel, few enough for two blocks
// on a CU, so that one asks for memory while the other multiplies.
//
// 8192 rows of x times one 4096 x 4096 matrix take 86 us at BT 256 (3.2
// PFLOP/s; the instructions alone would take 27): two blocks follow each
// other on a CU, and the first stage's requests, the results' way out and the
// operand reads that the products do not cover stand beside the products.
// 24576 routes over 256 matrices of 2048 x 4096 (1.1 GB) take 310 us at BT
// 128, 3.7 TB/s: bound by the matrices' bytes and, from L2, the routes'.  At
// BT 64, one route to each of some 200 of them take 152 us, 5.7 TB/s.
// A second stage on its way to registers took 379 us (BT 128, for want of
// registers) and 150 (BT 64; 21.3 for 20.8 where 45 MB are read).
constexpr int tile_rows(int bt) { return bt == 256 ? 256 : 128; }
typedef float f32x16 __attribute__((ext_vector_type(16)));

// The scales of two stages (16 blocks) of a row, from block b0; past the
// row's last block 0.  VEC: 16, rows are whole aligned 16-byte vectors; 4,
// whole dwords; 1, neither: a load for each byte, and at 128 and 256 routes
// more registers than there are (76 to 108 bytes a lane in scratch), which
// costs up to half of the rate (k 2944 / 2880, us: 256 matrices of 2048 rows
// for 96 routes each 267 / 517, for 12 each 186 / 255; one 4096 x k for 8192
// rows 100 / 203).
template <int VEC>
__device__ __forceinline__ u32x4 load_scales(const uint8_t *row, int b0, int nblk) {
    u32x4 v;
    if constexpr (VEC == 16) {
        v = *reinterpret_cast<const u32x4 *>(row + min(b0, nblk - 16));   // past the last: never read
    } else {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int b = b0 + 4 * d;
            if constexpr (VEC == 4) {
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
    }
    return v;
}

template <int N> struct Tiles {
    static constexpr int n = N;
};

template <int BT, bool SWIGLU, int SVEC, typename OUT>
__global__ __launch_bounds__(kThreads, BT == 256 ? 1 : 2) void mx_tile_kernel(
    MxParams p, const uint8_t *__restrict__ xc, const uint8_t *__restrict__ xs, const int32_t *__restrict__ n_runs,
    const Run *__restrict__ runs, const int32_t *__restrict__ routes, int R, int max_runs, int row_tiles,
    FastDiv by_K, OUT *__restrict__ out) {
    constexpr int kTileRows = tile_rows(BT);
    constexpr int kAcross = BT == 256 ? 2 : 4;       // waves along the rows; the others along the routes
    constexpr int kWaveRows = kTileRows / kAcross, kWaveRoutes = BT * kAcross / kWaves;
    constexpr int kN = kWaveRows / 32, kT = kWaveRoutes / 32;
    constexpr int kWLoads = kTileRows / 32, kXLoads = BT / 32;
    constexpr bool kSkip = BT < 256;                 // route tiles past the run are left out
    // scales are kept two stages of all rows at a time: matrix rows, then routes
    constexpr int kSLoads = (kTileRows + BT + kThreads - 1) / kThreads;
    struct Stages {
        uint8_t w[2][kTileRows * kStageBytes], x[2][BT * kStageBytes];
        uint8_t sc[2][kSLoads * kThreads][2 * kStageBlocks];
    };
    __shared__ __align__(16) uint8_t lds[sizeof(Stages)];
    Stages &buf = *reinterpret_cast<Stages *>(lds);
    auto &wbuf = buf.w;
    auto &xbuf = buf.x;
    auto &sc = buf.sc;

    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int c = lane & 31, h = lane / 32;
    // Consecutive workgroups go to the eight XCDs in turn: a run's row tiles
    // go to one of them, one behind the other, so that its L2 holds their
    // routes' x.  (The run is read beside the number of runs; past it there
    // is room in the table, but nothing that is used.)
    const int ri = (int)(blockIdx.x / 8) / row_tiles * 8 + (int)(blockIdx.x % 8);
    const int tile = (int)(blockIdx.x / 8) % row_tiles;
    if (ri >= max_runs) return;
    Run run;
    if (n_runs != nullptr) {
        const int n = n_runs[0];
        run = runs[ri];
        if (ri >= n) return;
    } else {
        run = Run{0, ri * BT, min(BT, R - ri * BT), 0};
    }

    const int cols = SWIGLU ? p.n / 2 : p.n;
    constexpr int kCols = SWIGLU ? kTileRows / 2 : kTileRows;   // output columns of the block
    const int j0 = tile * kCols;
    const int nblk = p.k / 32, stages = (nblk + kStageBlocks - 1) / kStageBlocks;
    const int64_t row_bytes = (int64_t)nblk * 16;
    // LDS row r of the weights: with SwiGLU each wave's rows are gate rows,
    // then the same number of up rows
    auto matrix_row = [&](int r) -> int64_t {
        if constexpr (SWIGLU) {
            constexpr int kHalf = kWaveRows / 2;
            const int j = min(j0 + r / kWaveRows * kHalf + r % kHalf, cols - 1);
            return (int64_t)run.row * p.n + (r % kWaveRows >= kHalf ? cols : 0) + j;
        } else {
            return (int64_t)run.row * p.n + min(j0 + r, cols - 1);
        }
    };
    // the run's routes, the last repeated past its end
    __shared__ int32_t list[BT];
    if (tid < BT) {
        const int at = run.start + min(tid, run.count - 1);
        list[tid] = n_runs != nullptr ? routes[at] : at;
    }
    lds_barrier();

    const int wn = wave % kAcross, wt = wave / kAcross;
    const int live = run.count - wt * kWaveRoutes;   // the wave's routes in the run
    f32x16 acc[kN][kT];
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < kT; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

    if (run.row >= 0) {
        const uint8_t *wp[kWLoads], *xp[kXLoads];
        const int lr = tid / 8, chunk = (tid & 7) ^ ((lr >> 1) & 7);
#pragma unroll
        for (int i = 0; i < kWLoads; ++i) wp[i] = p.codes + matrix_row(32 * i + lr) * row_bytes;
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) xp[i] = xc + (int64_t)by_K(list[32 * i + lr]) * row_bytes;
        const uint8_t *sp[kSLoads];
#pragma unroll
        for (int i = 0; i < kSLoads; ++i) {
            const int r = tid + i * kThreads;
            sp[i] = r < kTileRows ? p.scales + matrix_row(r) * nblk
                                  : xs + (int64_t)by_K(list[min(r - kTileRows, BT - 1)]) * nblk;
        }
        u32x4 sr[kSLoads];
        auto scales_fetch = [&](int g) {
#pragma unroll
            for (int i = 0; i < kSLoads; ++i) sr[i] = load_scales<SVEC>(sp[i], g * 2 * kStageBlocks, nblk);
        };
        auto scales_put = [&](int b) {
#pragma unroll
            for (int i = 0; i < kSLoads; ++i) *reinterpret_cast<u32x4 *>(sc[b][tid + i * kThreads]) = sr[i];
        };

        const int r0 = wn * kWaveRows + c, t0 = wt * kWaveRoutes + c;
        // all of k with the wave's first NT route tiles (and, kSkip, the
        // block's first 32 NT routes alone)
        auto all_stages = [&](auto tiles) {
            constexpr int NT = decltype(tiles)::n, kX = kSkip ? NT : kXLoads;
            // what a thread moves in a stage: a part of the next stage from
            // its register to LDS, and the same part of the stage after that
            // from memory to the register
            constexpr int kMoves = kWLoads + kX, kProducts = 4 * kN * NT, kReads = kN + NT;
            u32x4 part[kMoves];
            auto from_memory = [&](int i, int st) {      // stages past the last repeat it
                const int off = min(min(st, stages - 1) * kStageBlocks + chunk, nblk - 1) * 16;
                part[i] = *reinterpret_cast<const u32x4 *>((i < kWLoads ? wp[i < kWLoads ? i : 0]
                                                                        : xp[i < kWLoads ? 0 : i - kWLoads]) + off);
            };
            auto to_lds = [&](int i, int b) {
                uint8_t *to = i < kWLoads ? &wbuf[b][i * 4096] : &xbuf[b][(i - kWLoads) * 4096];
                *reinterpret_cast<u32x4 *>(to + tid * 16) = part[i];
            };
            // Stage st from buffer b = st & 1, into which the stage after next
            // goes once all have read it; the next goes to the other buffer,
            // the scales of the next two stages in every second stage.
            //
            // A wave issues in order, and a request to memory can hold it up
            // for a hundred cycles, an LDS access for tens.  So the moves and
            // the operand reads of the next step are set between the matrix
            // instructions, of 32 cycles each, one or two at a time, and kept
            // there (sched_barrier): with all requests before the products a
            // stage of BT 256 took 6100 cycles, 2050 of them products.
            auto stage = [&](int b, int st) {
                const int g = (st >> 1) & 1;
                uint32_t sa[kN], sb[NT];
                u32x4 wa[2][kN], xb[2][NT];
                auto read = [&](int e, int s) {          // operand e of step s
                    const int slot = ((4 * h + s) ^ ((c >> 1) & 7)) * 16;
                    if (e < NT)
                        xb[s & 1][e < NT ? e : 0] =
                            *reinterpret_cast<const u32x4 *>(&xbuf[b][(t0 + 32 * e) * kStageBytes + slot]);
                    else
                        wa[s & 1][e < NT ? 0 : e - NT] =
                            *reinterpret_cast<const u32x4 *>(&wbuf[b][(r0 + 32 * (e - NT)) * kStageBytes + slot]);
                };
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    sb[i] = *reinterpret_cast<const uint32_t *>(
                        &sc[g][kTileRows + t0 + 32 * i][kStageBlocks * b + 4 * h]);
#pragma unroll
                for (int i = 0; i < kN; ++i)
                    sa[i] = *reinterpret_cast<const uint32_t *>(&sc[g][r0 + 32 * i][kStageBlocks * b + 4 * h]);
#pragma unroll
                for (int e = 0; e < kReads; ++e) read(e, 0);
#define MOE_STEP(S)                                                                                              \
    _Pragma("unroll") for (int m = 0; m < kN * NT; ++m) {                                                        \
        const int i = m / NT, j = m % NT, at = S * kN * NT + m;                                                  \
        __builtin_amdgcn_sched_barrier(0);                                                                       \
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(wa[S & 1][i]), widen(xb[S & 1][j]),   \
                                                                    acc[i][j], kFp4, kFp4, S, (int)sa[i], S,    \
                                                                    (int)sb[j]);                                 \
        if (S < 3) {                                                                                             \
            _Pragma("unroll") for (int e = 0; e < kReads; ++e)                                                   \
                if (e * kN * NT / kReads == m) read(e, S + 1);                                                   \
        }                                                                                                        \
        _Pragma("unroll") for (int t = 0; t < kMoves; ++t)                                                       \
            if (t * kProducts / kMoves == at) {                                                                  \
                to_lds(t, b ^ 1);                                                                                \
                from_memory(t, st + 2);                                                                          \
            }                                                                                                    \
        if ((!kSkip || b == 1) && at == kProducts - 1) {                                                         \
            scales_put(g ^ 1);                                                                                   \
            scales_fetch(((st + 1) >> 1) + 1);                                                                   \
        }                                                                                                        \
    }
                MOE_STEP(0)
                MOE_STEP(1)
                MOE_STEP(2)
                MOE_STEP(3)
#undef MOE_STEP
                __builtin_amdgcn_sched_barrier(0);
                lds_barrier();
            };

            scales_fetch(0);
#pragma unroll
            for (int i = 0; i < kMoves; ++i) from_memory(i, 0);
            scales_put(0);
#pragma unroll
            for (int i = 0; i < kMoves; ++i) to_lds(i, 0);
            scales_fetch(1);
#pragma unroll
            for (int i = 0; i < kMoves; ++i) from_memory(i, 1);
            lds_barrier();
            if constexpr (kSkip) {
                for (int st = 0; st < stages; st += 2) {
                    stage(0, st);
                    if (st + 1 >= stages) break;
                    stage(1, st + 1);
                }
            } else {
                // (two copies of the stage would not fit the registers: the
                // scales are put and fetched again in the second)
#pragma unroll 1
                for (int st = 0; st < stages; ++st) stage(st & 1, st);
            }
        };
        if constexpr (kSkip) {
            static_assert(kT <= 4, "route tiles of a wave");
            if (live > 96)
                all_stages(Tiles<kT>{});
            else if (live > 64)
                all_stages(Tiles<(kT < 3 ? kT : 3)>{});
            else if (live > 32)
                all_stages(Tiles<2>{});
            else
                all_stages(Tiles<1>{});
        } else {
            all_stages(Tiles<kT>{});
        }
    }

    // The results go through LDS (the stages are done with it), so that whole
    // rows are written: lane (c, h) holds four columns each of 64 places, of
    // a route of its own.  Written from the registers they took a third of
    // the kernel's time at BT 256.  fp32 results of BT 256 go in two halves.
    constexpr int kPitch = kCols * (int)sizeof(OUT) + 16;
    constexpr int kPasses = BT * kPitch <= (int)sizeof(Stages) ? 1 : kWaves / kAcross;
    constexpr int kPassRoutes = BT / kPasses;
    static_assert(kPassRoutes * kPitch <= (int)sizeof(Stages) && (kPasses == 1 || kPassRoutes == kWaveRoutes), "LDS");
    constexpr int kUnits = kCols * (int)sizeof(OUT) / 16, kPerUnit = 16 / (int)sizeof(OUT);
    const bool whole = cols % kPerUnit == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
        if (pass > 0) lds_barrier();             // the first half has been read
        if (kPasses == 1 || wt == pass) {
#pragma unroll
            for (int j = 0; j < kT; ++j) {
                const int at = (kPasses == 1 ? wt * kWaveRoutes : 0) + 32 * j + c;
                // groups of four rows: 4 kN of them, with SwiGLU the first half gate, the second up
                constexpr int kGroups = SWIGLU ? 2 * kN : 4 * kN;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int col = wn * (kCols / kAcross) + 8 * g + 4 * h;
                    f32x4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = acc[g / 4][j][4 * (g % 4) + e];
                        if constexpr (SWIGLU) {
                            constexpr int kUp = 2 * kN;
                            v[e] = silu(v[e]) * acc[(g + kUp) / 4][j][4 * ((g + kUp) % 4) + e];
                        }
                    }
                    uint8_t *to = lds + at * kPitch + col * (int)sizeof(OUT);
                    if constexpr (sizeof(OUT) == 4)
                        *reinterpret_cast<f32x4 *>(to) = v;
                    else
                        *reinterpret_cast<uint2 *>(to) = uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
                }
            }
        }
        lds_barrier();
        const int n = min(run.count - pass * kPassRoutes, kPassRoutes);
        if (whole) {
            for (int i = tid; i < n * kUnits; i += kThreads) {
                const int t = i / kUnits, col = i % kUnits * kPerUnit;
                if (j0 + col >= cols) continue;
                *reinterpret_cast<u32x4 *>(out + (int64_t)list[pass * kPassRoutes + t] * cols + j0 + col) =
                    *reinterpret_cast<const u32x4 *>(lds + t * kPitch + col * (int)sizeof(OUT));
            }
        } else {
            for (int i = tid; i < n * kCols; i += kThreads) {
                const int t = i / kCols, col = i % kCols;
                if (j0 + col >= cols) continue;
                out[(int64_t)list[pass * kPassRoutes + t] * cols + j0 + col] =
                    *reinterpret_cast<const OUT *>(lds + t * kPitch + col * (int)sizeof(OUT));
            }
        }
    }
}

}  // namespace

size_t mx_workspace_bytes(int P, int n, int k, int T, int K) {
    (void)n;
    return mx_ws(P, k, T, K).total;
}

namespace {

// Blocks of the many-block form that keep the device busy; with fewer, k is
// split over the waves instead (split / many, us: 64 blocks 4.7 / 9.1, 256
// 11.3 / 10.7, 320 8.4 / 9.9, 384 27.5 / 32.0, 512 19.6 / 15.2 and 24.9 /
// 16.4, 1024 33.9 / 33.0).  A coarse rule: between 64 and 512 the two cross
// more than once, as k and the lists decide too; the worst of these costs 6 %.
constexpr int64_t kManyBlocks = 512;
// Blocks for the passes over one matrix row's list, where lists may be long:
// the longest list of a skewed batch is the kernel's last block.  1200 routes
// over 160 matrices of 512 x 1024 in 1, 2, 4 blocks (us): evenly spread 15.4
// 15.8 19.2, 50 more on one matrix 26.3 19.4 19.8, 200 67.8 39.5 28.8.
constexpr int kPassBlocks = 2;

template <bool SWIGLU, bool INLINE>
hipError_t launch_stream_shape(const MxParams &p, int mode, const int32_t *n_runs, const Run *runs,
                               const int32_t *routes, int R, int64_t slots, hipStream_t s) {
    const int cols = p.swiglu ? p.n / 2 : p.n;
    const bool x_vec = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.x_stride % 8 == 0;
    const uintptr_t sp = reinterpret_cast<uintptr_t>(p.scales);
    const int block_cols = kWaves * (SWIGLU ? 1 : 2) * kTile;
    const int wide = (cols + block_cols - 1) / block_cols, passes = mode == kByRow ? kPassBlocks : 1;
    if (wide * slots >= kManyBlocks) {
        const dim3 grid((unsigned)(wide * slots * passes));
#define MOE_STREAM(VEC)                                                                                        \
    hipLaunchKernelGGL((mx_stream_kernel<SWIGLU, VEC, INLINE>), grid, dim3(kThreads), 0, s, p, mode, x_vec,    \
                       (int)slots, passes, n_runs, runs, routes, R)
        if (p.k % 256 == 0 && sp % 8 == 0)
            MOE_STREAM(true);
        else
            MOE_STREAM(false);
#undef MOE_STREAM
    } else {
        const dim3 grid((cols + kTile - 1) / kTile, (unsigned)slots);
#define MOE_SPLIT(U, VEC)                                                                                       \
    hipLaunchKernelGGL((mx_split_kernel<SWIGLU, U, VEC, INLINE>), grid, dim3(kThreads), 0, s, p, mode, x_vec, \
                       n_runs, runs, routes, R)
        // four steps at once where each of the four waves has that many (2 / 4
        // steps, us: k 2048 5.13 / 4.85, 4096 6.65 / 6.20, 8192 10.1 / 9.5)
        if (p.k % 512 == 0 && p.k >= 2048 && sp % 16 == 0)
            MOE_SPLIT(4, true);
        else if (p.k % 256 == 0 && sp % 8 == 0)
            MOE_SPLIT(2, true);
        else
            MOE_SPLIT(2, false);
#undef MOE_SPLIT
    }
    return hipGetLastError();
}

hipError_t launch_stream(const MxParams &p, int mode, const int32_t *n_runs, const Run *runs,
                         const int32_t *routes, int R, int64_t slots, hipStream_t s) {
    if (mode == kRuns)
        return p.swiglu ? launch_stream_shape<true, false>(p, mode, n_runs, runs, routes, R, slots, s)
                        : launch_stream_shape<false, false>(p, mode, n_runs, runs, routes, R, slots, s);
    return p.swiglu ? launch_stream_shape<true, true>(p, mode, n_runs, runs, routes, R, slots, s)
                    : launch_stream_shape<false, true>(p, mode, n_runs, runs, routes, R, slots, s);
}

template <int BT, typename OUT>
hipError_t launch_tile(const MxParams &p, const uint8_t *xc, const uint8_t *xs, const int32_t *n_runs,
                       const Run *runs, const int32_t *routes, int R, int64_t max_runs, hipStream_t s) {
    const int per = p.swiglu ? tile_rows(BT) / 2 : tile_rows(BT), cols = p.swiglu ? p.n / 2 : p.n;
    const int row_tiles = (cols + per - 1) / per;
    const unsigned grid = (unsigned)((max_runs + 7) / 8 * 8 * row_tiles);
    const FastDiv by_K(p.K, (uint64_t)R);
    const uintptr_t sp = reinterpret_cast<uintptr_t>(p.scales);
#define MOE_TILE(S, V)                                                                                          \
    hipLaunchKernelGGL((mx_tile_kernel<BT, S, V, OUT>), dim3(grid), dim3(kThreads), 0, s, p, xc, xs, n_runs, runs, \
                       routes, R, (int)max_runs, row_tiles, by_K, static_cast<OUT *>(p.out))
#define MOE_TILE_S(S)                        \
    if (p.k % 512 == 0 && sp % 16 == 0)      \
        MOE_TILE(S, 16);                     \
    else if (p.k % 128 == 0 && sp % 4 == 0)  \
        MOE_TILE(S, 4);                      \
    else                                     \
        MOE_TILE(S, 1);
    if (p.swiglu) {
        MOE_TILE_S(true)
    } else {
        MOE_TILE_S(false)
    }
#undef MOE_TILE_S
#undef MOE_TILE
    return hipGetLastError();
}

// Routes a run may hold.  A longer run reads its matrix once for more routes
// and lets an operand byte from LDS meet more of the other; it costs idle
// columns where lists are shorter, and blocks.  Measured (us, n x k of one
// matrix, one product from bf16 x; "lists" are routes spread at random):
//   16 -> 64: the tile kernel needs a launch of its own before it but keeps
//     more of the matrix on its way.  67 MB of matrices in question, one
//     route each: 16.1 / 18.4 (1024 x 2048), 17.1 / 23.0 (2048 x 512), 18.5
//     / 16.5 (4096 x 4096); 100 MB 27.5 / 26.7; 134 MB 35.0 / 29.4; 33 MB
//     12.6 / 16.2.  By the mean, at 42 MB: 8 routes 16.0 / 18.8, 12 19.8 /
//     19.2, 16 28.8 / 19.3.  One matrix has no list longer than the mean:
//     32 routes 12.7 / 14.8, 48 18.0 / 16.3.
//   64 -> 128: mean 48 22.0 / 23.6, 56 26.9 / 24.0, 64 30.1 / 24.4; fewer
//     blocks than CUs: 256 routes of one 8192 x 4096 28.1 / 33.0, 1024 (512
//     blocks) 53.6 / 39.5.
//   128 -> 256 (32 matrices, 2048 rows): k 4096 mean 256 101 / 109, 512 168
//     / 164, 1024 294 / 277; k 1024 mean 512 69 / 77; one 8192 x 4096, 1024
//     routes (128 blocks) 39.5 / 51.5, 4096 (512) 141 / 111.
int run_length_for(const MxParams &p, int R) {
    constexpr int64_t kMuch = 80 << 20;      // bytes of matrices in question
    constexpr int kCus = 256;
    const bool lists = p.idx != nullptr;
    const int matrices = lists ? std::min(R, p.P) : 1, mean = R / matrices;
    auto blocks = [&](int len) {
        const int rows = tile_rows(len);
        return std::max<int64_t>(matrices, R / len) * ((p.n + rows - 1) / rows);
    };
    if (mean >= 384 && p.k >= 2048 && blocks(256) >= kCus) return 256;
    if (mean >= 56 && blocks(128) >= kCus) return 128;
    if (mean >= (lists ? 12 : 48) || (int64_t)matrices * p.n * p.k / 2 >= kMuch) return 64;
    return kTile;
}

// Runs the lists may hold.
int64_t max_runs_of(const MxParams &p, int R, int run_length) {
    return p.idx != nullptr ? std::min<int64_t>(R, (int64_t)p.P + 1) + R / run_length
                            : (R + run_length - 1) / run_length;
}

template <typename OUT>
hipError_t launch_tile_for(int run_length, const MxParams &p, const uint8_t *xc, const uint8_t *xs,
                           const int32_t *n_runs, const Run *runs, const int32_t *routes, int R,
                           int64_t max_runs, hipStream_t s) {
    if (run_length == 256) return launch_tile<256, OUT>(p, xc, xs, n_runs, runs, routes, R, max_runs, s);
    if (run_length == 128) return launch_tile<128, OUT>(p, xc, xs, n_runs, runs, routes, R, max_runs, s);
    return launch_tile<64, OUT>(p, xc, xs, n_runs, runs, routes, R, max_runs, s);
}

}  // namespace

bool mx_launchable(const MxParams &p) {
    const int R = p.T * p.K;
    if (R == 0) return true;
    const int run_length = run_length_for(p, R);
    const int cols = p.swiglu ? p.n / 2 : p.n;
    // (the short runs' narrowest block that comes in numbers: a wave's columns times four)
    const int width = run_length == kTile ? kWaves * (p.swiglu ? 1 : 2) * kTile
                                          : tile_rows(run_length) / (p.swiglu ? 2 : 1);
    const int64_t tiles = (cols + width - 1) / width;
    return (max_runs_of(p, R, run_length) + 8) * tiles * kPassBlocks <= (int64_t)UINT32_MAX / kThreads;
}

hipError_t launch_mx_product(const MxParams &p, int *list_length, hipStream_t s) {
    const int R = p.T * p.K;
    if (R == 0) return hipSuccess;
    const MxWs L = mx_ws(p.P, p.k, p.T, p.K);
    int32_t *n_runs = reinterpret_cast<int32_t *>(p.ws + L.n_runs);
    Run *runs = reinterpret_cast<Run *>(p.ws + L.runs);
    int32_t *routes = reinterpret_cast<int32_t *>(p.ws + L.routes);
    uint8_t *xc = p.ws + L.codes, *xs = p.ws + L.scales;
    const int run_length = run_length_for(p, R);
    const bool stream = run_length == kTile;
    if (p.idx != nullptr && stream && R <= kInlineRoutes) {
        const bool by_route = R <= p.P;
        return launch_stream(p, by_route ? kByRoute : kByRow, nullptr, nullptr, nullptr, R,
                             by_route ? R : p.P + 1, s);
    }
    // lists of routes, and x quantised where a tile kernel reads it
    const int lists = p.idx != nullptr && *list_length != run_length;
    if (lists || !stream) {
        PrepareParams a{.idx = p.idx,
                        .R = R,
                        .P = p.P,
                        .run_length = run_length,
                        .lists = lists,
                        .staged = 0,
                        .n_runs = n_runs,
                        .runs = runs,
                        .routes = routes,
                        .x = p.x,
                        .x_stride = p.x_stride,
                        .units = stream ? 0 : (int64_t)p.T * (p.k / kPer),
                        .upr = p.k / kPer,
                        .by_upr = FastDiv((uint64_t)p.k / kPer, (uint64_t)p.T * (p.k / kPer)),
                        .codes = xc,
                        .scales = xs};
        size_t lds = lists ? (2 * kGroupWaves + (size_t)p.P + 1) * 4 : 0;
        if (lists && lds + (size_t)R * 4 <= kPrepareLds) {
            a.staged = 1;
            lds += (size_t)R * 4;
        }
        const bool vec = vector_rows(p.x, p.x_stride, p.T, 2);
        const void *fn = vec ? reinterpret_cast<const void *>(&mx_prepare_kernel<true>)
                             : reinterpret_cast<const void *>(&mx_prepare_kernel<false>);
        if (lds > 65536) {
            hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, kPrepareLds);
            if (e != hipSuccess) return e;
        }
        const unsigned grid = lists + (unsigned)std::min<int64_t>((a.units + kGroupThreads - 1) / kGroupThreads, 4096);
        if (vec)
            hipLaunchKernelGGL(mx_prepare_kernel<true>, dim3(grid), dim3(kGroupThreads), lds, s, a);
        else
            hipLaunchKernelGGL(mx_prepare_kernel<false>, dim3(grid), dim3(kGroupThreads), lds, s, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (lists) *list_length = run_length;
    }
    const int64_t max_runs = max_runs_of(p, R, run_length);
    if (p.idx == nullptr) n_runs = nullptr;
    if (stream) return launch_stream(p, kRuns, n_runs, runs, routes, R, max_runs, s);
    return p.out_type == MOE_TYPE_F32
               ? launch_tile_for<float>(run_length, p, xc, xs, n_runs, runs, routes, R, max_runs, s)
               : launch_tile_for<uint16_t>(run_length, p, xc, xs, n_runs, runs, routes, R, max_runs, s);
}

}  // namespace moe
