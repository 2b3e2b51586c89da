// Lists of routes by matrix row: a stable counting sort of [T K] ids.
//
//   order   the route numbers sorted by their row, ascending within a row;
//           routes without a row (id outside [0, P)) come last
//   offsets [P + 1] the place of each row's first route; offsets[P] is the
//           place of the first route without a row
//
// A route's place is the number of routes of smaller rows, plus the number of
// earlier routes of its row.  The second is counted in pieces: routes of
// earlier blocks, of earlier waves of the block, of the wave's earlier
// routes, and of lower lanes (ballots over the bits of the row), so the order
// hangs on no atomic.  Each wave has a stretch of the piece and its own
// counts of it in LDS; where those do not fit (many rows), the waves take 64
// routes each in turn, a barrier between them (20000 routes: 16 barriers for
// each 1024, 1.2 us).
//
// Up to kOneBlock routes one block does all; above, a launch counts each
// piece's routes and a second places them, each block summing the counts of
// the pieces before it.  Bound by latency: 2 x 4 bytes a route are read and
// 4 written (163840 routes over 512 rows, 2 MB: 2.4 + 11.6 us; one token's 8
// over 256 3.1).
#include <algorithm>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
// Routes that one block sorts alone (256 rows, us: 2400 routes by one block
// 12.8, by two 7.5; 8000 16.5 and 8.1).
constexpr int kOneBlock = 2048;
// Pieces: every block reads the counts of all of them, pieces x (P + 1) words,
// 0.05 us a piece, and takes 0.85 us for each 1024 of its own routes: about
// the square root of R / 64 is best (163840 routes over 512 rows, us: 160
// pieces 19.5, 80 14.5, 40 13.5; 24576 over 256: 12 8.3, 6 10.5).  Of more
// rows than waves count alone, fewer.
constexpr int kMaxPieces = 256, kMaxPiecesWide = 32;
constexpr int kAhead = 20;          // counts of a row on their way together
constexpr int kHeld = 4;            // ids a lane holds, requested together
constexpr int kMaxOwnRows = 4095;   // rows of which each wave has counts of its own
static_assert(kListsMaxRoutes / kMaxPieces <= 65535, "a piece's counts in 16 bits");

struct ListsShape {
    int pieces, per;
};
ListsShape lists_shape(int P, int64_t R) {
    if (R <= kOneBlock) return {1, kOneBlock};
    const int most = P > kMaxOwnRows ? kMaxPiecesWide : kMaxPieces;
    int64_t pieces = 1;
    while (pieces < most && (pieces + 1) * (pieces + 1) <= R / 64) ++pieces;
    const int64_t per = ((R + pieces - 1) / pieces + kThreads - 1) / kThreads * kThreads;
    return {(int)((R + per - 1) / per), (int)per};
}

__device__ __forceinline__ int row_of(int id, int P) { return id >= 0 && id < P ? id : P; }

// Lanes of the wave whose row equals this lane's (lanes out of play: row P + 1).
__device__ __forceinline__ uint64_t same_row(int row, int bits) {
    uint32_t lo = ~0u, hi = ~0u;
    for (int b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((row >> b) & 1);
        const uint32_t flip = (uint32_t)((row >> b & 1) - 1);   // all ones where the bit is 0
        lo &= (uint32_t)one ^ flip;
        hi &= (uint32_t)(one >> 32) ^ flip;
    }
    return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ int lanes_below(uint64_t m) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// Adds the rows of n ids to cnt, kHeld of a thread's ids on their way together.
__device__ __forceinline__ void count_rows(const int32_t *idx, int n, int P, int32_t *cnt) {
    for (int i0 = threadIdx.x; i0 < n; i0 += kHeld * kThreads) {
        int id[kHeld];
#pragma unroll
        for (int k = 0; k < kHeld; ++k) id[k] = idx[min(i0 + k * kThreads, n - 1)];
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            if (i0 + k * kThreads < n) atomicAdd(&cnt[row_of(id[k], P)], 1);
    }
}

__global__ __launch_bounds__(kThreads) void lists_count_kernel(const int32_t *__restrict__ idx, int R, int P, int per,
                                                               int32_t *__restrict__ counts) {
    extern __shared__ __align__(16) int32_t cnt[];
    for (int r = threadIdx.x; r <= P; r += kThreads) cnt[r] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * per;
    const int n = (int)min((int64_t)per, (int64_t)R - begin);
    count_rows(idx + begin, n, P, cnt);
    __syncthreads();
    int32_t *to = counts + (int64_t)blockIdx.x * (P + 1);
    for (int r = threadIdx.x; r <= P; r += kThreads) to[r] = cnt[r];
}

// pieces == 1: counts is not read, the block counts for itself.
__global__ __launch_bounds__(kThreads) void lists_place_kernel(const int32_t *__restrict__ idx, int R, int P, int per,
                                                               int pieces, int bits,
                                                               const int32_t *__restrict__ counts,
                                                               int32_t *__restrict__ offsets,
                                                               int32_t *__restrict__ order) {
    extern __shared__ __align__(16) int32_t lds[];
    int32_t *wsum = lds;             // [kWaves]
    int32_t *total = lds + kWaves;   // [P + 1]: routes of each row, then the next free place
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int64_t begin = (int64_t)blockIdx.x * per;
    const int n = (int)min((int64_t)per, (int64_t)R - begin);

    // the wave's stretch of the piece, its first ids on their way at once
    const int stretch = per / kWaves, w0 = wave * stretch, w1 = min(w0 + stretch, n);
    int held[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) held[k] = n > 0 ? idx[begin + min(w0 + k * kWave + lane, n - 1)] : 0;

    if (pieces == 1) {
        for (int r = tid; r <= P; r += kThreads) total[r] = 0;
        __syncthreads();
        count_rows(idx, n, P, total);
        __syncthreads();
    }
    // Exclusive prefix sum over the rows, kThreads of them at a time; for
    // several pieces, plus the row's routes in earlier pieces.
    int before = 0;
    for (int base = 0; base <= P; base += kThreads) {
        const int r = base + tid;
        int all = 0, mine = 0;
        if (r <= P) {
            if (pieces == 1) {
                all = total[r];
            } else {
                for (int b0 = 0; b0 < pieces; b0 += kAhead) {
                    int v[kAhead];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) v[i] = counts[(int64_t)min(b0 + i, pieces - 1) * (P + 1) + r];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        all += b0 + i < pieces ? v[i] : 0;
                        mine += b0 + i < (int)blockIdx.x ? v[i] : 0;
                    }
                }
            }
        }
        const int incl = wave_inclusive_sum(all);
        if (lane == kWave - 1) wsum[wave] = incl;
        __syncthreads();
        int off = before, sum = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int v = wsum[w];
            off += w < wave ? v : 0;
            sum += v;
        }
        const int start = off + incl - all;
        if (r <= P) {
            total[r] = start + mine;
            if (blockIdx.x == 0) offsets[r] = start;
        }
        before += sum;
        __syncthreads();
    }

    if (P <= kMaxOwnRows) {
        // counts of each wave's stretch, then where it begins in each row
        uint16_t *own = reinterpret_cast<uint16_t *>(total + P + 1), *mine = own + wave * (P + 1);
        for (int i = tid; i < kWaves * (P + 1); i += kThreads) own[i] = 0;
        __syncthreads();
        // 64 routes: a lane's row (13 bits), how many of lower lanes and of all
        // lanes have the same (7 bits each)
        auto match = [&](int i0, int id) {
            const int row = i0 + lane < w1 ? row_of(id, P) : P + 1;
            const uint64_t same = same_row(row, bits);
            return (uint32_t)row | (uint32_t)lanes_below(same) << 13 | (uint32_t)__popcll(same) << 20;
        };
        static_assert(kMaxOwnRows + 1 < 1 << 13, "a row in 13 bits");
        auto count = [&](int i0, uint32_t m) {
            const int row = m & 0x1fff;
            if (i0 + lane < w1 && (m >> 13 & 127) == 0) mine[row] = (uint16_t)(mine[row] + (m >> 20));
            __builtin_amdgcn_wave_barrier();
        };
        auto put = [&](int i0, uint32_t m) {
            const int row = m & 0x1fff, rank = m >> 13 & 127;
            if (i0 + lane < w1) {
                const int at = mine[row];
                order[total[row] + at + rank] = (int32_t)(begin + i0 + lane);
                __builtin_amdgcn_wave_barrier();
                if (rank == 0) mine[row] = (uint16_t)(at + (m >> 20));
            }
            __builtin_amdgcn_wave_barrier();
        };
        const int late = w0 + kHeld * kWave;   // past what is held: matched in both passes
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            if (w0 + k * kWave < w1) {
                held[k] = (int)match(w0 + k * kWave, held[k]);
                count(w0 + k * kWave, held[k]);
            }
        for (int i0 = late; i0 < w1; i0 += kWave) count(i0, match(i0, idx[begin + min(i0 + lane, n - 1)]));
        __syncthreads();
        for (int r = tid; r <= P; r += kThreads) {
            int at = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int v = own[w * (P + 1) + r];
                own[w * (P + 1) + r] = (uint16_t)at;
                at += v;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            if (w0 + k * kWave < w1) put(w0 + k * kWave, held[k]);
        for (int i0 = late; i0 < w1; i0 += kWave) put(i0, match(i0, idx[begin + min(i0 + lane, n - 1)]));
        return;
    }
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        const bool live = i < n;
        const int row = live ? row_of(idx[begin + i], P) : P + 1;
        const uint64_t same = same_row(row, bits);
        const int rank = lanes_below(same);
        int place = 0;
        for (int w = 0; w < kWaves; ++w) {
            if (w == wave && live) {
                place = total[row] + rank;
                __builtin_amdgcn_wave_barrier();
                if (rank == 0) total[row] = place + __popcll(same);
            }
            __syncthreads();
        }
        if (live) order[place] = (int32_t)(begin + i);
    }
}

size_t place_lds(int P) {
    return (size_t)(kWaves + P + 1) * 4 + (P <= kMaxOwnRows ? (size_t)kWaves * (P + 1) * 2 : 0);
}

}  // namespace

size_t lists_workspace_bytes(int P, int64_t R) {
    const ListsShape s = lists_shape(P, R);
    return s.pieces == 1 ? 0 : (size_t)s.pieces * (P + 1) * 4;
}

hipError_t launch_lists(const int32_t *idx, int R, int P, int32_t *offsets, int32_t *order, int32_t *counts,
                        hipStream_t s) {
    const ListsShape sh = lists_shape(P, R);
    const size_t lds = place_lds(P);
    if (lds > 65536) {   // always the largest, so that calls from two threads agree
        const int most = (int)std::max(place_lds(kListsMaxRows), place_lds(kMaxOwnRows));
        for (const void *k : {reinterpret_cast<const void *>(&lists_place_kernel),
                              reinterpret_cast<const void *>(&lists_count_kernel)}) {
            hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, most);
            if (e != hipSuccess) return e;
        }
    }
    int bits = 1;
    while ((1 << bits) <= P + 1) ++bits;
    if (sh.pieces > 1)
        hipLaunchKernelGGL(lists_count_kernel, dim3(sh.pieces), dim3(kThreads), lds, s, idx, R, P, sh.per, counts);
    hipLaunchKernelGGL(lists_place_kernel, dim3(sh.pieces), dim3(kThreads), lds, s, idx, R, P, sh.per, sh.pieces, bits,
                       counts, offsets, order);
    return hipGetLastError();
}

}  // namespace moe
