// Lists of routes by matrix row: a stable counting sort of [T K] ids.
//
//   order   the route numbers sorted by their row, ascending within a row;
//           routes without a row (id outside [0, P)) come last
//   offsets [P + 1] the place of each row's first route; offsets[P] is the
//           place of the first route without a row
//
// A route's place is the number of routes of smaller rows, plus the number of
// earlier routes of its row.  The second is counted in pieces: routes of
// earlier blocks, of earlier waves of the block (the waves take turns), and
// of lower lanes of the wave (ballots over the bits of the row), so the order
// hangs on no atomic.
//
// Up to kOneBlock routes one block does all; above, a launch counts each
// piece's routes and a second places them, each block summing the counts of
// the pieces before it.  Bound by latency: 2 x 4 bytes a route are read and
// 4 written (163840 routes: 2 MB).
#include <algorithm>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
// Routes that one block sorts alone.
constexpr int kOneBlock = 8192;
// Routes of a piece, and the most pieces: every block reads the counts of all
// pieces before its own, pieces x (P + 1) words.
constexpr int kPiece = 2048;
constexpr int kMaxPieces = 256, kWideRows = 2048, kMaxPiecesWide = 32;

struct ListsShape {
    int pieces, per;
};
ListsShape lists_shape(int P, int64_t R) {
    if (R <= kOneBlock) return {1, kOneBlock};
    const int most = P > kWideRows ? kMaxPiecesWide : kMaxPieces;
    const int64_t want = (R + kPiece - 1) / kPiece;
    const int64_t pieces = std::min<int64_t>(want, most);
    const int64_t per = ((R + pieces - 1) / pieces + kThreads - 1) / kThreads * kThreads;
    return {(int)((R + per - 1) / per), (int)per};
}

__device__ __forceinline__ int row_of(int id, int P) { return id >= 0 && id < P ? id : P; }

// Lanes of the wave whose row equals this lane's (lanes out of play: row P + 1).
__device__ __forceinline__ uint64_t same_row(int row, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((row >> b) & 1);
        m &= (row >> b) & 1 ? one : ~one;
    }
    return m;
}

__device__ __forceinline__ int lanes_below(uint64_t m) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

__global__ __launch_bounds__(kThreads) void lists_count_kernel(const int32_t *__restrict__ idx, int R, int P, int per,
                                                               int32_t *__restrict__ counts) {
    extern __shared__ __align__(16) int32_t cnt[];
    for (int r = threadIdx.x; r <= P; r += kThreads) cnt[r] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * per;
    const int n = (int)min((int64_t)per, (int64_t)R - begin);
    for (int i = threadIdx.x; i < n; i += kThreads) atomicAdd(&cnt[row_of(idx[begin + i], P)], 1);
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

    if (pieces == 1) {
        for (int r = tid; r <= P; r += kThreads) total[r] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) atomicAdd(&total[row_of(idx[i], P)], 1);
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
#pragma unroll 8
                for (int b = 0; b < pieces; ++b) {
                    const int v = counts[(int64_t)b * (P + 1) + r];
                    all += v;
                    mine += b < (int)blockIdx.x ? v : 0;
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

size_t place_lds(int P) { return (size_t)(kWaves + P + 1) * 4; }

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
        const int most = (int)place_lds(kListsMaxRows);
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
