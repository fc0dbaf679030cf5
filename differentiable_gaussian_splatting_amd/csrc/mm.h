// mm.h -- the matrix product under the layer and Muon kernels: one block's
// tile of C[m][n] = sum over k of A[m][k] B[n][k], on the matrix cores.
//
// Operands.  Each is a matrix in memory whose k either runs along the rows
// ("row": value (r, k) at p[r ld + k]) or down the columns ("col": at
// p[k ld + r]), so that x w^T, dz w and dz^T x all read their operands where
// they are: nothing is transposed in memory.  A thread loads 8 values of k
// (row), or 8 x 4 values (col) that it turns round in registers, and writes
// them to LDS as 16-byte chunks of consecutive k, the form that a lane of the
// matrix instruction takes.
//
// Types.  16-bit values are multiplied as they are (products are exact in f32,
// sums are f32).  f32 values are split into parts whose products run at the
// 16-bit rate, 16 times that of f32 matrix instructions:
//   P = 3: x = h + m + l in bf16, each the rounding of what the ones before
//          leave (2^-8 of it at most, so 2^-24 |x| is left out).  Six products
//          are kept (h h, h m, m h, m m, h l, l h); all that is left out of
//          x y is below 2^-22 |x y|, and typically 2^-26.  Any f32 range; a
//          value that is not finite makes its results NaN.
//   P = 2: x s = h + l in f16 with a power of two s that the caller knows to
//          keep |x s| below 65504 (2^-22 |x s| is left out while |x s| >= 2^-3,
//          2^-25 below that).  Three products (h h, h l, l h).  For the
//          Newton-Schulz products, whose values are bounded.
//
// LDS holds each tile as rows of BK values; chunk c of row r stands at place
// c ^ f(r), f from the low four bits of r, so that the 16 lanes that read one
// chunk of 16 rows, and the lanes that write chunks of every fourth row, meet
// different banks.  A tile's successor is loaded into registers while the
// matrix instructions run and is written to the other LDS buffer afterwards
// (one barrier per BK).
#pragma once

#include "gs_tensor.h"

namespace gsm {

using gst::bf16;
using gst::f16;

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct Operand {
    const void* p;
    int64_t ld;
    int64_t rows;     // rows (row) or columns (col) that exist; beyond them the last one is read
    float scale;      // P = 2: power of two
    int32_t gate;     // > 0: row r of the tile is a gate or an up row (see row_of_tile)
};

template <int BM_, int BN_, int BK_, int WM_, int WN_, int STAGES_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, STAGES = STAGES_;
    static constexpr int NT = WM * WN * 64;
    static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;   // 16 x 16 results of a wave
    static_assert(BM % (WM * 16) == 0 && BN % (WN * 16) == 0 && BK % 32 == 0, "tile");
};

template <typename S, int P>
struct Part;
template <>
struct Part<f16, 1> { typedef f16 E; };
template <>
struct Part<bf16, 1> { typedef bf16 E; };
template <>
struct Part<float, 2> { typedef f16 E; };
template <>
struct Part<float, 3> { typedef bf16 E; };

__device__ __forceinline__ f32x4 mfma(gst::Pack<bf16, 8> a, gst::Pack<bf16, 8> b, f32x4 c)
{
    typedef bf16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(gst::Pack<f16, 8> a, gst::Pack<f16, 8> b, f32x4 c)
{
    typedef f16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
}

// the P parts of 8 values
template <typename S, int P>
__device__ __forceinline__ void split(const S (&v)[8], float scale, gst::Pack<typename Part<S, P>::E, 8> (&out)[P])
{
    typedef typename Part<S, P>::E E;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (P == 1) {
            out[0].v[j] = v[j];
        } else {
            float x = P == 2 ? v[j] * scale : v[j];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const E e = (E)x;
                out[p].v[j] = e;
                x -= (float)e;
            }
        }
    }
}

// place of chunk c in row r of an LDS tile
template <int BK>
__device__ __forceinline__ int place(int r, int c)
{
    if constexpr (BK == 64) return c ^ ((r & 7) ^ ((r >> 3) & 1));
    else return c ^ (((r >> 1) & 3) ^ ((r >> 3) & 1));
}

// The matrix row that row r of a tile starting at n0 stands for.  With
// gate = F > 0 the tile alternates 16 gate rows (of [0, F)) and the 16 up rows
// of the same columns (F later), so that a wave holds both results of a column.
__device__ __forceinline__ int64_t row_of_tile(const Operand& o, int64_t n0, int r)
{
    if (o.gate == 0) return min(n0 + r, o.rows - 1);
    const int64_t f = n0 / 2 + (r >> 5) * 16 + (r & 15);
    return min(f, (int64_t)o.gate - 1) + ((r >> 4) & 1) * (int64_t)o.gate;
}

// One operand's way from memory to LDS: R rows of BK values per step.
template <typename S, int P, int R, int BK, int NT, bool COL>
struct Stage {
    typedef typename Part<S, P>::E E;
    static constexpr int kChunks = BK / 8;
    static constexpr int kUnits = COL ? R * BK / 32 : R * BK / 8;
    static constexpr int kPer = (kUnits + NT - 1) / NT;
    static constexpr bool kExact = kUnits % NT == 0;
    const S* at[kPer];    // the unit's first value at k = 0
    int64_t ld;
    int edge;             // COL: bit u: unit u reaches over the last column
    int64_t left[COL ? kPer : 1];
    float scale;
    S v[kPer][COL ? 8 : 1][COL ? 4 : 8];

    __device__ __forceinline__ bool mine(int u) const { return kExact || (int)threadIdx.x + u * NT < kUnits; }

    __device__ __forceinline__ void init(const Operand& o, int64_t r0)
    {
        ld = o.ld;
        edge = 0;
        scale = o.scale;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int id = (threadIdx.x + u * NT) % (kExact ? 1 << 30 : kUnits);
            if constexpr (COL) {
                const int64_t r = r0 + (id % (R / 4)) * 4;
                const int64_t c = min(r, o.rows - 1);
                at[u] = (const S*)o.p + (int64_t)(id / (R / 4)) * 8 * ld + c;
                left[u] = o.rows - 1 - c;      // columns after it
                if (left[u] < 3) edge |= 1 << u;
            } else {
                at[u] = (const S*)o.p + row_of_tile(o, r0, id / kChunks) * ld + (id % kChunks) * 8;
            }
        }
    }

    // the values of k in [k, k + BK); TAIL: those from kend on are zero
    template <bool TAIL>
    __device__ __forceinline__ void load(int64_t k, int64_t kend)
    {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            if (!mine(u)) continue;
            const int id = threadIdx.x + u * NT;
            if constexpr (COL) {
                const int64_t kk = k + (id / (R / 4)) * 8;
                const S* p = at[u] + k * ld;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (TAIL && kk + q >= kend) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[u][q][j] = (S)0.0f;
                    } else if (!((edge >> u) & 1)) {
                        const gst::Pack<S, 4> x = gst::load<S, 4>(p + q * ld);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[u][q][j] = x.v[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[u][q][j] = p[q * ld + min((int64_t)j, left[u])];
                    }
                }
            } else {
                const int64_t kk = k + (id % kChunks) * 8;
                const S* p = at[u] + k;
                if (!TAIL || kk + 8 <= kend) {
                    const gst::Pack<S, 8> x = gst::load<S, 8>(p);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[u][0][j] = x.v[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[u][0][j] = kk + j < kend ? p[j] : (S)0.0f;
                }
            }
        }
    }

    // to LDS: plane p of the tile at lds + p R BK
    __device__ __forceinline__ void commit(E* lds) const
    {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            if (!mine(u)) continue;
            const int id = threadIdx.x + u * NT;
#pragma unroll
            for (int j = 0; j < (COL ? 4 : 1); ++j) {
                S x[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) x[q] = COL ? v[u][COL ? q : 0][COL ? j : 0] : v[u][0][COL ? 0 : q];
                const int r = COL ? (id % (R / 4)) * 4 + j : id / kChunks;
                const int c = COL ? id / (R / 4) : id % kChunks;
                gst::Pack<E, 8> part[P];
                split<S, P>(x, scale, part);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    *reinterpret_cast<gst::Pack<E, 8>*>(__builtin_assume_aligned(
                        lds + p * R * BK + r * BK + place<BK>(r, c) * 8, 16)) = part[p];
            }
        }
    }
};

template <typename S, int P, typename T>
struct alignas(16) Lds {
    typedef typename Part<S, P>::E E;
    E b[T::STAGES][P * T::BN * T::BK];
    E a[T::STAGES][P * T::BM * T::BK];
};

// acc[i][j] += the 16 x 16 results of the calling wave: row j's m is its
// lane's (lane & 15), column i's n its lane's 4 (lane >> 4) + 0..3.
template <typename S, int P, bool ACOL, bool BCOL, typename T>
__device__ __forceinline__ void mm_tile(const Operand& A, const Operand& B, int64_t m0, int64_t n0, int64_t k0,
                                        int64_t k1, Lds<S, P, T>& lds, f32x4 (&acc)[T::NI][T::MI])
{
    typedef typename Part<S, P>::E E;
    constexpr int BK = T::BK;
    if (k0 >= k1) return;
    Stage<S, P, T::BM, BK, T::NT, ACOL> sa;
    Stage<S, P, T::BN, BK, T::NT, BCOL> sb;
    sa.init(A, m0);
    sb.init(B, n0);
    auto load = [&](int64_t k) {
        if (k + BK <= k1) {
            sb.template load<false>(k, k1);
            sa.template load<false>(k, k1);
        } else {
            sb.template load<true>(k, k1);
            sa.template load<true>(k, k1);
        }
    };
    load(k0);
    sb.commit(lds.b[0]);
    sa.commit(lds.a[0]);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int am = (wave % T::WM) * T::MI * 16 + (lane & 15), bn = (wave / T::WM) * T::NI * 16 + (lane & 15);
    int buf = 0;
    for (int64_t k = k0; k < k1; k += BK) {
        __syncthreads();
        const bool more = k + BK < k1;
        if (more) load(k + BK);
        const E *la = lds.a[buf], *lb = lds.b[buf];
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk) {
            gst::Pack<E, 8> fa[P][T::MI], fb[P][T::NI];
            const int ca = place<BK>(am, kk * 4 + (lane >> 4)) * 8, cb = place<BK>(bn, kk * 4 + (lane >> 4)) * 8;
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int i = 0; i < T::NI; ++i)
                    fb[p][i] = *reinterpret_cast<const gst::Pack<E, 8>*>(
                        __builtin_assume_aligned(lb + p * T::BN * BK + (bn + i * 16) * BK + cb, 16));
#pragma unroll
                for (int j = 0; j < T::MI; ++j)
                    fa[p][j] = *reinterpret_cast<const gst::Pack<E, 8>*>(
                        __builtin_assume_aligned(la + p * T::BM * BK + (am + j * 16) * BK + ca, 16));
            }
#pragma unroll
            for (int i = 0; i < T::NI; ++i)
#pragma unroll
                for (int j = 0; j < T::MI; ++j) {
                    if constexpr (P == 3) {
                        acc[i][j] = mfma(fb[2][i], fa[0][j], acc[i][j]);
                        acc[i][j] = mfma(fb[0][i], fa[2][j], acc[i][j]);
                        acc[i][j] = mfma(fb[1][i], fa[1][j], acc[i][j]);
                    }
                    if constexpr (P >= 2) {
                        acc[i][j] = mfma(fb[1][i], fa[0][j], acc[i][j]);
                        acc[i][j] = mfma(fb[0][i], fa[1][j], acc[i][j]);
                    }
                    acc[i][j] = mfma(fb[0][i], fa[0][j], acc[i][j]);
                }
        }
        if constexpr (T::STAGES == 2) buf ^= 1;
        else __syncthreads();
        if (more) {
            sb.commit(lds.b[buf]);
            sa.commit(lds.a[buf]);
        }
    }
}

// Tile t of tm x tn: in groups of eight rows of tiles, down the rows first, so
// that blocks that run together share operands' tiles.
__device__ __forceinline__ void tile_at(int64_t t, int64_t tm, int64_t tn, int64_t& i, int64_t& j)
{
    constexpr int64_t G = 8;
    const int64_t g = t / (G * tn), rows = min(G, tm - g * G), in = t - g * G * tn;
    i = g * G + in % rows;
    j = in / rows;
}

// Block b of n as a place in the order of tiles: neighbouring blocks go to
// different XCDs (b % 8), so that each XCD walks a range of its own and its
// L2 serves that range's tiles.
__device__ __forceinline__ int64_t xcd_order(int64_t b, int64_t n)
{
    const int64_t x = b & 7, each = n >> 3, more = n & 7;
    return x * each + min(x, more) + (b >> 3);
}

}  // namespace gsm
