// Products of bf16 rows with matrices of a pool bank (bf16, E2M1 or MXFP4),
// the rows grouped by matrix, on gfx950's bf16 matrix instructions.
//
// Places 0..R-1 are cut by offsets into groups; group g's places take matrix
// M = W[matrices[g]], [n][k]:
//   y = M x[place] + bias,   out[place] = act(y) (+ residual)
// with act one of the identity, silu, gelu, or (two halves of y) silu(gate)
// * up.  A dense product is the same with one group of all places.
//
// 4-bit weights are expanded to bf16 exactly (an E2M1 value times an E4M3
// value has at most six significant bits; times a power of two, two); an
// E2M1 matrix's global scale multiplies the fp32 sum.  Sums are fp32 in the
// matrix instructions; bias, activation and residual are applied to them in
// fp32 and rounded once, to the output's type.
#include <algorithm>

#include "k_rows.inc"

namespace moe {
namespace {

using namespace rows_detail;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
// 16 bytes at any element's address (global loads take unaligned addresses).
struct __attribute__((packed, aligned(2))) Bytes16 {
    uint32_t v[4];
};

constexpr int kTile = 16;        // rows and places of one 16 x 16 x 32 instruction
constexpr int kSlab = 128;       // elements of k in four of them

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ u32x4 load16(const void *p) {
    const Bytes16 b = *static_cast<const Bytes16 *>(p);
    return u32x4{b.v[0], b.v[1], b.v[2], b.v[3]};
}

// Eight elements from element e of a row of k, zeros past its end.
__device__ __forceinline__ u32x4 load8_tail(const uint16_t *row, int e, int k) {
    if (e + 8 <= k) return load16(row + e);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (e + i < k) v[i / 2] |= (uint32_t)row[e + i] << (16 * (i & 1));
    return v;
}

// A barrier that orders LDS alone: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// 32 consecutive weights of a 4-bit row to bf16, as four operands: two E2M1
// values a byte, even elements in the low nibble.  scale: two E4M3 bytes
// (elements 0-15 and 16-31), or one E8M0 byte.
template <int FMT> __device__ __forceinline__ u32x4 expand8(uint32_t word, uint32_t scale, int i) {
    u32x4 o;
    if constexpr (FMT == MOE_FMT_MXFP4) {
        const float s = e8m0_f(scale);
#define MOE_CVT(B) \
    o[B] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, s, B));
        MOE_CVT(0)
        MOE_CVT(1)
        MOE_CVT(2)
        MOE_CVT(3)
#undef MOE_CVT
    } else {
        const float s = e4m3_f(i < 2 ? scale & 0xffu : scale >> 8);
        // the products are exact in bf16: their upper halves are the values
#define MOE_CVT(B)                                                                                             \
    {                                                                                                          \
        const f32x2 f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, B);                               \
        o[B] = __builtin_amdgcn_perm(__float_as_uint(f.y * s), __float_as_uint(f.x * s), 0x07060302u);         \
    }
        MOE_CVT(0)
        MOE_CVT(1)
        MOE_CVT(2)
        MOE_CVT(3)
#undef MOE_CVT
    }
    return o;
}
template <int FMT> constexpr int scale_block() { return FMT == MOE_FMT_E2M1 ? 16 : 32; }

// ------------------------------------------------------------------ groups

// A piece of a group: its matrix and its places [start, start + count).
struct Piece {
    int group, start, count;
};

// Piece number `slot` of the groups cut into pieces of `length` places, found
// by one wave: each lane counts four groups' pieces, 256 groups at a time.
// false: there are fewer.  (All of a wave's lanes take part; the answer is
// the same in each.)
__device__ __forceinline__ bool find_piece(const int32_t *offsets, int G, int R, int length, int slot, Piece &out) {
    if (offsets == nullptr) {
        out = Piece{0, slot * length, min(length, R - slot * length)};
        return out.count > 0;
    }
    const int lane = threadIdx.x & (kWave - 1);
    int before = 0;
    for (int base = 0; base < G; base += 4 * kWave) {
        const int g0 = base + 4 * lane;
        int o[5], n[4], mine = 0;
#pragma unroll
        for (int i = 0; i < 5; ++i) o[i] = min(max(offsets[min(g0 + i, G)], 0), R);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            n[i] = g0 + i < G ? (max(o[i + 1] - o[i], 0) + length - 1) / length : 0;
            mine += n[i];
        }
        const int incl = wave_inclusive_sum(mine);
        const uint64_t here = __ballot(before + incl > slot);
        if (here != 0) {
            const int who = __ffsll((unsigned long long)here) - 1;
            int left = slot - (before + incl - mine), i = 0;
            for (; i < 3 && left >= n[i]; ++i) left -= n[i];
            // (only lane `who` holds a meaningful i)
            const int at = i == 0 ? o[0] : i == 1 ? o[1] : i == 2 ? o[2] : o[3];
            const int end = i == 0 ? o[1] : i == 1 ? o[2] : i == 2 ? o[3] : o[4];
            const int start = at + left * length;
            out.group = __builtin_amdgcn_readlane(g0 + i, who);
            out.start = __builtin_amdgcn_readlane(start, who);
            out.count = __builtin_amdgcn_readlane(min(length, end - start), who);
            return true;
        }
        before += __builtin_amdgcn_readlane(incl, kWave - 1);
    }
    return false;
}

// The most pieces that groups of R places can have.
int64_t max_pieces(const ProductParams &p, int length) {
    if (p.offsets == nullptr) return (p.R + length - 1) / length;
    return std::min<int64_t>(p.G, p.R) + p.R / length;
}

// The matrix of a group, -1 where it has none.
__device__ __forceinline__ int matrix_of(const ProductParams &p, int group) {
    const int m = p.matrices != nullptr ? p.matrices[group] : group;
    return m >= 0 && m < p.P ? m : -1;
}

// The row of x a place reads and the row of out it writes; a place whose
// gathered or scattered row is not there is left out (out -1).
struct Place {
    int in, out;
};
__device__ __forceinline__ Place place_at(const ProductParams &p, int i) {
    Place at{i, i};
    if (p.gather != nullptr) at.in = p.gather[i];
    if (p.scatter != nullptr) at.out = p.scatter[i];
    at.in = at.in < 0 ? -1 : at.in / p.gather_div;
    if (at.in < 0 || at.in >= p.x_rows) {
        at.in = 0;
        at.out = -1;
    }
    if (at.out >= p.out_rows) at.out = -1;
    return at;
}

// ------------------------------------------------------------------ epilogue

__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

__device__ __forceinline__ float load_any(const void *base, int type, int64_t i) {
    return type == MOE_TYPE_F32 ? static_cast<const float *>(base)[i] : bf16_f(static_cast<const uint16_t *>(base)[i]);
}

// Four consecutive outputs col.. of row `row`: y (and, for SWIGLU, the up
// half's u) are sums.  whole: rows start on whole vectors of four outputs
// (and residuals) and cols is a multiple of 4.
template <bool SWIGLU>
__device__ __forceinline__ void finish4(const ProductParams &p, int mat, int row, int col, int cols, bool whole, f32x4 y,
                                        f32x4 u) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int j = min(col + e, cols - 1);
        float a = y[e], b = u[e];
        if (p.bias != nullptr) {
            a += load_any(p.bias, p.bias_type, (int64_t)mat * p.n + j);
            if constexpr (SWIGLU) b += load_any(p.bias, p.bias_type, (int64_t)mat * p.n + cols + j);
        }
        if constexpr (SWIGLU)
            a = silu(a) * b;
        else if (p.act == MOE_ACT_SILU)
            a = silu(a);
        else if (p.act == MOE_ACT_GELU)
            a = 0.5f * a * (1.f + erff(a * 0.70710678118654752f));
        v[e] = a;
    }
    if (p.residual != nullptr) {
        const int64_t at = (int64_t)row * p.res_stride + col;
        if (whole && p.res_type == MOE_TYPE_BF16) {
            if (col < cols) {
                const uint2 r = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.residual) + at);
                v[0] += bf16_lo(r.x), v[1] += bf16_hi(r.x), v[2] += bf16_lo(r.y), v[3] += bf16_hi(r.y);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < cols) v[e] += load_any(p.residual, p.res_type, at + e);
        }
    }
    const int64_t at = (int64_t)row * p.out_stride + col;
    if (p.out_type == MOE_TYPE_F32) {
        float *o = static_cast<float *>(p.out) + at;
        if (whole) {
            if (col < cols) *reinterpret_cast<f32x4 *>(o) = f32x4{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < cols) o[e] = v[e];
        }
    } else {
        uint16_t *o = static_cast<uint16_t *>(p.out) + at;
        if (whole) {
            if (col < cols) *reinterpret_cast<uint2 *>(o) = uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < cols) o[e] = f32_to_bf16(v[e]);
        }
    }
}

// Four zeros in the place of a row whose group has no matrix.
__device__ __forceinline__ void zero4(const ProductParams &p, int row, int col, int cols) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (col + e >= cols) break;
        const int64_t at = (int64_t)row * p.out_stride + col + e;
        if (p.out_type == MOE_TYPE_F32)
            static_cast<float *>(p.out)[at] = 0.f;
        else
            static_cast<uint16_t *>(p.out)[at] = 0;
    }
}

bool whole_vectors(const ProductParams &p, int cols) {
    auto fits = [&](const void *base, int type, int64_t stride) {
        const int bytes = type == MOE_TYPE_F32 ? 4 : 2;
        return reinterpret_cast<uintptr_t>(base) % (4 * bytes) == 0 && stride % 4 == 0;
    };
    return cols % 4 == 0 && fits(p.out, p.out_type, p.out_stride) &&
           (p.residual == nullptr || fits(p.residual, p.res_type, p.res_stride));
}

// ------------------------------------------------------------------ few rows

// 32 weights of a row from element e, and their scale bytes.
template <int FMT> struct Weights {
    u32x4 v[FMT == MOE_FMT_BF16 ? 4 : 1];
    uint32_t scale = 0;
    // whole: all 32 are inside the row
    __device__ __forceinline__ void load(const ProductParams &p, int64_t row, int e, bool whole) {
        if constexpr (FMT == MOE_FMT_BF16) {
            const uint16_t *src = reinterpret_cast<const uint16_t *>(p.w) + row * p.k;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = whole ? load16(src + e + 8 * i) : load8_tail(src, e + 8 * i, p.k);
        } else {
            v[0] = u32x4{0, 0, 0, 0};
            scale = 0;
            if (whole || e < p.k) {
                v[0] = *reinterpret_cast<const u32x4 *>(p.w + row * (p.k / 2) + e / 2);
                if constexpr (FMT == MOE_FMT_E2M1)
                    scale = *reinterpret_cast<const uint16_t *>(p.scales + row * (p.k / 16) + e / 16);
                else
                    scale = p.scales[row * (p.k / 32) + e / 32];
            }
        }
    }
    __device__ __forceinline__ u32x4 operand(int i) const {
        if constexpr (FMT == MOE_FMT_BF16)
            return v[i];
        else
            return expand8<FMT>(v[0][i], scale, i);
    }
};

// A block's waves share M tiles of 16 rows of one matrix (SWIGLU: a tile of
// gate and one of up rows) and up to 16 NB places, and split k: each takes
// every WAVES-th slab of 128.  Lane l = 16 q + c holds, of matrix row c and
// of place c, the 32 elements from 32 q of a slab: k is permuted alike in
// both operands, which leaves the sums as they are, and every load is a whole
// vector.  The waves' sums are added in LDS, in wave order.
template <int FMT, bool SWIGLU, int M, int NB, int WAVES, int U>
__global__ __launch_bounds__(WAVES *kWave) void product_split_kernel(ProductParams p, int tiles, bool whole_out) {
    static_assert(!SWIGLU || M % 2 == 0, "gate and up tiles");
    __shared__ __align__(16) f32x4 red[WAVES][M * NB][kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int c = lane & (kTile - 1), q = lane / kTile;
    constexpr int kOut = SWIGLU ? M / 2 : M;           // tiles of output columns
    const int cols = SWIGLU ? p.n / 2 : p.n;
    const int j0 = (int)(blockIdx.x % tiles) * kOut * kTile;
    Piece piece;
    if (!find_piece(p.offsets, p.G, p.R, kTile * NB, (int)(blockIdx.x / tiles), piece)) return;
    const int mat = matrix_of(p, piece.group);
    Place at[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        at[b] = place_at(p, piece.start + min(b * kTile + c, piece.count - 1));
        if (b * kTile + c >= piece.count) at[b].out = -1;
    }
    if (mat < 0) {
        for (int t = wave; t < kOut * NB; t += WAVES) {
            int out = -1;
#pragma unroll
            for (int i = 0; i < NB; ++i) out = i == t % NB ? at[i].out : out;
            if (out >= 0) zero4(p, out, j0 + (t / NB) * kTile + 4 * q, cols);
        }
        return;
    }
    int64_t wrow[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int j = min(j0 + (m % kOut) * kTile + c, cols - 1);
        wrow[m] = (int64_t)mat * p.n + (m >= kOut ? cols : 0) + j;
    }
    const uint16_t *xr[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) xr[b] = p.x + (int64_t)at[b].in * p.x_stride;

    f32x4 acc[M][NB];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[m][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int full = p.k / kSlab;
    // whole slabs, U of them on their way together (past the last, the last again)
    for (int s0 = wave; s0 < full; s0 += WAVES * U) {
        Weights<FMT> w[U][M];
        u32x4 xv[U][NB][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = min(s0 + u * WAVES, full - 1) * kSlab + 32 * q;
#pragma unroll
            for (int m = 0; m < M; ++m) w[u][m].load(p, wrow[m], e, true);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[u][b][i] = load16(xr[b] + e + 8 * i);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u * WAVES >= full) break;
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x4 a = w[u][m].operand(i);
#pragma unroll
                    for (int b = 0; b < NB; ++b) acc[m][b] = mfma16(a, xv[u][b][i], acc[m][b]);
                }
        }
    }
    if (p.k % kSlab != 0 && wave == full % WAVES) {    // the last, partial slab
        const int e = full * kSlab + 32 * q;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            Weights<FMT> w;
            w.load(p, wrow[m], e, false);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4 a = w.operand(i);
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[m][b] = mfma16(a, load8_tail(xr[b], e + 8 * i, p.k), acc[m][b]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) red[wave][m * NB + b][lane] = acc[m][b];
    __syncthreads();
    const float glob = FMT == MOE_FMT_E2M1 && p.globals != nullptr ? p.globals[mat] : 1.f;
#pragma unroll
    for (int t0 = 0; t0 < kOut * NB; t0 += WAVES) {
        const int t = t0 + wave;
        if (t >= kOut * NB) break;
        f32x4 y = red[0][t][lane], u = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 1; w < WAVES; ++w) y += red[w][t][lane];
        if constexpr (SWIGLU) {
            u = red[0][t + kOut * NB][lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) u += red[w][t + kOut * NB][lane];
        }
        if constexpr (FMT == MOE_FMT_E2M1) {
            y *= glob;
            u *= glob;
        }
        const int b = t % NB;
        int out = -1;
#pragma unroll
        for (int i = 0; i < NB; ++i) out = i == b ? at[i].out : out;
        const int col = j0 + t / NB * kTile + 4 * q;
        if (out >= 0 && col < cols) finish4<SWIGLU>(p, mat, out, col, cols, whole_out, y, u);
    }
}

template <int FMT, bool SWIGLU, int NB>
hipError_t launch_split(const ProductParams &p, hipStream_t s) {
    constexpr int M = SWIGLU ? 2 : 1, kWaves = 8, U = FMT == MOE_FMT_BF16 ? (NB == 4 ? 1 : 2) : (NB == 4 ? 1 : 4);
    constexpr int kCols = (SWIGLU ? M / 2 : M) * kTile;
    const int cols = SWIGLU ? p.n / 2 : p.n, tiles = (cols + kCols - 1) / kCols;
    const dim3 grid((unsigned)(tiles * max_pieces(p, kTile * NB)));
    hipLaunchKernelGGL((product_split_kernel<FMT, SWIGLU, M, NB, kWaves, U>), grid, dim3(kWaves * kWave), 0, s, p,
                       tiles, whole_vectors(p, cols));
    return hipGetLastError();
}

template <int FMT> hipError_t launch_format(const ProductParams &p, hipStream_t s) {
    return p.act == MOE_ACT_SWIGLU ? launch_split<FMT, true, 1>(p, s) : launch_split<FMT, false, 1>(p, s);
}

}  // namespace

bool product_launchable(const ProductParams &p) {
    const int64_t tiles = (p.n + kTile - 1) / kTile;
    return tiles * max_pieces(p, kTile) < (1ll << 32) / (8 * kWave);
}

hipError_t launch_product(const ProductParams &p, hipStream_t s) {
    switch (p.fmt) {
        case MOE_FMT_BF16: return launch_format<MOE_FMT_BF16>(p, s);
        case MOE_FMT_E2M1: return launch_format<MOE_FMT_E2M1>(p, s);
        default: return launch_format<MOE_FMT_MXFP4>(p, s);
    }
}

}  // namespace moe
