// mm.h -- the matrix product under the layer and Muon kernels: one block's
// tile of C[m][n] = sum over k of A[m][k] B[n][k], on the matrix cores.
//
// Operands.  Each is a matrix in memory whose k either runs along the rows
// ("row": value (r, k) at p[r ld + k]) or down the columns ("col": at
// p[k ld + r]), so that x w^T, dz w and dz^T x all read their operands where
// they are: nothing is transposed in memory.  A thread loads 8 neighbouring
// values and writes them to LDS as one 16-byte chunk.  A lane of the matrix
// instruction takes 8 consecutive k of one r: a chunk of a row tile, or two
// transposing LDS reads of a col tile, in which each group of 16 lanes fetches
// 4 k x 16 r and every lane receives its r's 4 values.
//
// Types.  16-bit values are multiplied as they are (products are exact in f32,
// sums are f32).  f32 values are split into parts whose products run at the
// 16-bit rate, 16 times that of f32 matrix instructions:
//   P = 3: x = h + m + l in bf16, each the rounding of what the ones before
//          leave (2^-8 of it at most, so 2^-24 |x| is left out).  Six products
//          are kept (h h, h m, m h, m m, h l, l h); all that is left out of
//          x y is below 2^-22 |x y|, and typically 2^-26.  Any f32 range, but a
//          value that is infinite or above bf16's largest makes its results NaN
//          (the layers sum those again, sum_again in layer_mm.h).
//   P = 2: x s = h + l in f16 with a power of two s that the caller knows to
//          keep |x s| below 65504 (2^-22 |x s| is left out while |x s| >= 2^-3,
//          2^-25 below that).  Three products (h h, h l, l h).  For the
//          Newton-Schulz products, whose values are bounded.
//
// LDS holds a row tile as rows of BK values, with chunk c of row r at place
// c ^ f(r), f from the low four bits of r: the 16 lanes that read one chunk of
// 16 rows meet different banks.  It holds a col tile as BK rows of R values,
// with 16-value unit q of row k at place q ^ h(k), so that the 16 rows of k
// that a transposing read touches spread over the banks.  A tile's successor
// is on its way while the matrix instructions run, to the other LDS buffer (one
// barrier per BK): 16-bit operands whose rows start on 16 bytes are loaded into
// LDS directly (Direct), others through registers (Stage), which also move
// values at the operands' edges and split f32 ones.
#pragma once

#include <type_traits>

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

// BM x BN results of WM x WN waves, BK values of k a step, in STAGES LDS buffers
template <int BM_, int BN_, int BK_, int WM_, int WN_, int STAGES_, bool TINY_ = false>
struct Tile {
    static constexpr bool TINY = TINY_;   // operands with fewer than 8 values of k or columns (see Stage)
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

// place of chunk c in row r of a row tile
template <int BK>
__device__ __forceinline__ int place(int r, int c)
{
    if constexpr (BK >= 64) return c ^ ((r & 7) ^ ((r >> 3) & 1));
    else return c ^ (((r >> 1) & 3) ^ ((r >> 3) & 1));
}
// what is xored into the 16-value unit of row k of a col tile of R values
template <int R>
__device__ __forceinline__ int unit_swap(int k)
{
    return ((k & 3) | ((k >> 1) & 4)) & (R / 16 - 1);
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

// v moved down by n places (zeros follow), n >= 0
__device__ __forceinline__ void move_down(float (&v)[8], int n)
{
#pragma unroll
    for (int step = 4; step; step >>= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = n & step ? (j + step < 8 ? v[j + step < 8 ? j + step : 0] : 0.0f) : v[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = n >= 8 ? 0.0f : v[j];
}
template <typename S>
__device__ __forceinline__ void move_down(S (&v)[8], int n)
{
    uint64_t lo, hi;
    __builtin_memcpy(&lo, &v[0], 8);
    __builtin_memcpy(&hi, &v[4], 8);
    if (n >= 4) {
        lo = hi;
        hi = 0;
    }
    const int bits = (n & 3) * 16;
    lo = n >= 8 ? 0 : (lo >> bits) | (hi << 1 << (63 - bits));
    hi = hi >> bits;
    __builtin_memcpy(&v[0], &lo, 8);
    __builtin_memcpy(&v[4], &hi, 8);
}

// One operand's way from memory to LDS: R rows (or columns) of BK values per
// step, in units of 8 neighbouring values of k (row) or r (col).  A unit that
// would reach over the end of k or over the last column is read from 8 values
// before that end and moved down in its registers: one load either way.  So
// there have to be 8 values of k (row) or 8 columns (col); TINY tiles, for
// operands that have fewer, read value by value instead.
template <typename S, int P, int R, int BK, int NT, bool COL, bool TINY>
struct Stage {
    typedef typename Part<S, P>::E E;
    static constexpr int kSide = (COL ? R : BK) / 8;   // units side by side
    static constexpr int kStep = NT / kSide;           // rows (of k, where col) from a thread's unit to its next
    static constexpr int kUnits = R * BK / 8;
    static constexpr int kPer = (kUnits + NT - 1) / NT;
    static constexpr bool kExact = kUnits % NT == 0;
    const S* at;          // the thread's first unit at k = 0
    const S* p;
    int64_t ld, rows, r0;
    float scale;
    int32_t gate;
    int32_t over;         // col: places that the thread's units reach over the last column
    S v[kPer][8];
    static_assert(NT % kSide == 0, "a thread's units share their columns");
    static_assert(COL || kStep % 32 == 0 || kPer == 1, "gate and up rows alternate by 16");

    __device__ __forceinline__ bool mine(int u) const { return kExact || (int)threadIdx.x + u * NT < kUnits; }
    __device__ __forceinline__ static int side() { return threadIdx.x % kSide; }
    __device__ __forceinline__ static int row(int u) { return threadIdx.x / kSide + u * kStep; }

    __device__ __forceinline__ void init(const Operand& o, int64_t tile0)
    {
        ld = o.ld;
        rows = o.rows;
        scale = o.scale;
        gate = o.gate;
        r0 = tile0;
        p = (const S*)o.p;
        over = 0;
        if constexpr (COL) {
            const int64_t r = r0 + side() * 8, from = TINY ? min(r, rows - 1) : min(r, rows - 8);
            over = (int)min((int64_t)8, TINY ? 8 - (rows - from) : r - from);
            at = p + (int64_t)row(0) * ld + from;
        } else {
            at = p + row_of_tile(o, r0, row(0)) * ld + side() * 8;
        }
    }

    // Loads the values of k in [k, k + BK).  EDGE: k + BK may lie behind kend,
    // and the tile may reach over the last row or column (what it holds there
    // is any of the operand's values).  Nothing here waits for what it loads.
    template <bool EDGE>
    __device__ __forceinline__ void load(int64_t k, int64_t kend)
    {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            if (!mine(u)) continue;
            if constexpr (COL) {
                const int64_t kk = EDGE ? min(k + row(u), kend - 1) - row(0) : k + u * kStep;
                if constexpr (TINY) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[u][j] = at[kk * ld + min(j, 7 - over)];
                } else {
                    take(v[u], at + kk * ld);
                }
            } else if constexpr (EDGE) {
                const int64_t kk = k + side() * 8;
                const Operand o = {nullptr, ld, rows, scale, gate};
                const S* q = p + row_of_tile(o, r0, row(u)) * ld + kk;
                if constexpr (TINY) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[u][j] = kk + j < kend ? q[j] : (S)0.0f;
                } else {
                    take(v[u], q - max(kk + 8 - kend, (int64_t)0));
                }
            } else {
                take(v[u], at + k + u * (gate ? kStep / 2 : kStep) * ld);
            }
        }
    }
    __device__ __forceinline__ static void take(S (&v)[8], const S* q)
    {
        const gst::Pack<S, 8> x = gst::load<S, 8>(q);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x.v[j];
    }

    // To LDS: plane p of the tile at lds + p R BK.  EDGE: with the values that
    // a unit has brought from before an end moved down, and zeros from `left`
    // values of k on.
    template <bool EDGE>
    __device__ __forceinline__ void commit(E* lds, int64_t left)
    {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            if (!mine(u)) continue;
            const int r = row(u), c = side();
            if constexpr (EDGE && COL) {
                if (r >= left) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[u][j] = (S)0.0f;
                } else if (!TINY && over) {
                    move_down(v[u], over);
                }
            } else if constexpr (EDGE && !TINY) {
                const int64_t n = c * 8 + 8 - left;
                if (n > 0) move_down(v[u], (int)min(n, (int64_t)8));
            }
            const int to = COL ? r * R + ((c >> 1) ^ unit_swap<R>(r)) * 16 + (c & 1) * 8 : r * BK + place<BK>(r, c) * 8;
            gst::Pack<E, 8> part[P];
            split<S, P>(v[u], scale, part);
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<gst::Pack<E, 8>*>(__builtin_assume_aligned(lds + p * R * BK + to, 16)) = part[p];
        }
    }
};

// The same way without registers, for whole tiles of a 16-bit operand whose rows
// start on 16 bytes: each lane's 16 bytes go straight to LDS, the wave's 64
// chunks to 1 KB in lane order, so the lane fetches the chunk that belongs to
// its place.  The compiler does not see these loads: done() waits for all of
// them (M0, which holds their LDS address, is reserved: no value lives in it).  (With the builtin for this load it waits for them before the next LDS
// read, whose buffer is another one, and the loads hide behind nothing: 256 x 256
// tiles 900 TFLOP/s, 990 this way; 128 x 128 790 and 890; through registers 915
// and 740.)
template <typename S, int R, int BK, int NT, bool COL>
struct Direct {
    static constexpr int kSide = (COL ? R : BK) / 8, kStep = NT / kSide, kPer = R * BK / 8 / NT;
    static_assert(NT % kSide == 0 && R * BK / 8 % NT == 0 && kStep % 16 == 0, "places repeat every 16 rows");
    const S* at;
    int64_t step;   // from a thread's chunk to its next

    __device__ __forceinline__ void init(const Operand& o, int64_t r0)
    {
        const int row = threadIdx.x / kSide, c = threadIdx.x % kSide;
        if constexpr (COL) {
            at = (const S*)o.p + (int64_t)row * o.ld + r0 + ((c >> 1) ^ unit_swap<R>(row)) * 16 + (c & 1) * 8;
            step = kStep * o.ld;
        } else {
            static_assert(kStep % 32 == 0, "gate and up rows alternate by 16");
            at = (const S*)o.p + row_of_tile(o, r0, row) * o.ld + place<BK>(row, c) * 8;
            step = (o.gate ? kStep / 2 : kStep) * o.ld;
        }
    }
    __device__ __forceinline__ void load(int64_t k, int64_t ld, S* lds) const
    {
        const S* p = at + (COL ? k * ld : k);
        S* const to = lds + (threadIdx.x >> 6) * 512;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const uint32_t m0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)(to + u * NT * 8);
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                         :
                         : "s"(__builtin_amdgcn_readfirstlane(m0)), "v"(p + u * step)
                         : "memory");
        }
    }
};
__device__ __forceinline__ void done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A wave's N blocks of 16 rows (columns) of a tile, as matrix operands.
template <typename E, int P, int R, int BK, int N, bool COL>
struct Fragments {
    int base[COL ? N : BK / 32];

    // r0: the wave's first row, a multiple of 16
    __device__ __forceinline__ void init(int r0, int lane)
    {
        if constexpr (COL) {
            const int k = (lane >> 4) * 8 + ((lane >> 2) & 3);
#pragma unroll
            for (int i = 0; i < N; ++i) base[i] = k * R + ((r0 / 16 + i) ^ unit_swap<R>(k)) * 16 + (lane & 3) * 4;
        } else {
            const int r = r0 + (lane & 15);
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk) base[kk] = r * BK + place<BK>(r, kk * 4 + (lane >> 4)) * 8;
        }
    }

    // block i at k = 32 kk of plane p
    __device__ __forceinline__ gst::Pack<E, 8> get(const E* lds, int p, int i, int kk) const
    {
        if constexpr (COL) {
            typedef short v4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) v4* at;
            const E* q = lds + p * R * BK + kk * 32 * R + base[i];
            const v4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at)q);
            const v4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at)(q + 4 * R));
            gst::Pack<E, 8> both;
            __builtin_memcpy(&both.v[0], &lo, 8);
            __builtin_memcpy(&both.v[4], &hi, 8);
            return both;
        } else {
            return *reinterpret_cast<const gst::Pack<E, 8>*>(
                __builtin_assume_aligned(lds + p * R * BK + base[kk] + i * 16 * BK, 16));
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
// WHOLE: the caller's tiles and k end with whole tiles and steps.  DIRECT: the
// rows of both operands start on 16 bytes.
template <typename S, int P, bool ACOL, bool BCOL, typename T, bool WHOLE = false, bool DIRECT = false>
__device__ __forceinline__ void mm_tile(const Operand& A, const Operand& B, int64_t m0, int64_t n0, int64_t k0,
                                        int64_t k1, Lds<S, P, T>& lds, f32x4 (&acc)[T::NI][T::MI])
{
    typedef typename Part<S, P>::E E;
    constexpr int BK = T::BK;
    if (k0 >= k1) return;
    Stage<S, P, T::BM, BK, T::NT, ACOL, T::TINY> sa;
    Stage<S, P, T::BN, BK, T::NT, BCOL, T::TINY> sb;
    sa.init(A, m0);
    sb.init(B, n0);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Fragments<E, P, T::BM, BK, T::MI, ACOL> fa;
    Fragments<E, P, T::BN, BK, T::NI, BCOL> fb;
    fa.init((wave % T::WM) * T::MI * 16, lane);
    fb.init((wave / T::WM) * T::NI * 16, lane);
    const int64_t bn = B.gate ? T::BN / 2 : T::BN, n1 = B.gate ? n0 / 2 : n0;
    const bool edge = m0 + T::BM > A.rows || n1 + bn > (B.gate ? B.gate : B.rows);
    int buf = 0;
    auto compute = [&]() {
        const E *la = lds.a[buf], *lb = lds.b[buf];
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk) {
            gst::Pack<E, 8> a[P][T::MI], b[P][T::NI];
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int i = 0; i < T::NI; ++i) b[p][i] = fb.get(lb, p, i, kk);
#pragma unroll
                for (int j = 0; j < T::MI; ++j) a[p][j] = fa.get(la, p, j, kk);
            }
#pragma unroll
            for (int i = 0; i < T::NI; ++i)
#pragma unroll
                for (int j = 0; j < T::MI; ++j) {
                    if constexpr (P == 3) {
                        acc[i][j] = mfma(b[2][i], a[0][j], acc[i][j]);
                        acc[i][j] = mfma(b[0][i], a[2][j], acc[i][j]);
                        acc[i][j] = mfma(b[1][i], a[1][j], acc[i][j]);
                    }
                    if constexpr (P >= 2) {
                        acc[i][j] = mfma(b[1][i], a[0][j], acc[i][j]);
                        acc[i][j] = mfma(b[0][i], a[1][j], acc[i][j]);
                    }
                    acc[i][j] = mfma(b[0][i], a[0][j], acc[i][j]);
                }
        }
    };
    // steps from `from` up to `to`, both loops' code apart: what the edges need
    // would cost the whole tiles' loop its registers
    auto steps = [&](auto is_edge, int64_t from, int64_t to) {
        constexpr bool EDGE = decltype(is_edge)::value;
        sb.template load<EDGE>(from, to);
        sa.template load<EDGE>(from, to);
        sb.template commit<EDGE>(lds.b[buf], to - from);
        sa.template commit<EDGE>(lds.a[buf], to - from);
        for (int64_t k = from; k < to; k += BK) {
            __syncthreads();
            const bool more = k + BK < to;
            if (more) {
                sb.template load<EDGE>(k + BK, to);
                sa.template load<EDGE>(k + BK, to);
            }
            compute();
            if constexpr (T::STAGES == 2) buf ^= 1;
            else __syncthreads();
            if (more) {
                sb.template commit<EDGE>(lds.b[buf], to - k - BK);
                sa.template commit<EDGE>(lds.a[buf], to - k - BK);
            }
        }
    };
    if constexpr (WHOLE) {
        steps(std::false_type{}, k0, k1);
        return;
    }
    const int64_t whole = edge ? k0 : k0 + (k1 - k0) / BK * BK;
    if constexpr (DIRECT) {
        static_assert(P == 1 && T::STAGES == 2 && BK == 64, "direct loads");
        Direct<S, T::BM, BK, T::NT, ACOL> da;
        Direct<S, T::BN, BK, T::NT, BCOL> db;
        da.init(A, m0);
        db.init(B, n0);
        // LDS reads of the second half of a step between the products of the first
        constexpr int kReads = T::MI * (ACOL ? 2 : 1) + T::NI * (BCOL ? 2 : 1), kProducts = T::MI * T::NI;
        auto next = [&](int64_t k) {
            db.load(k, B.ld, lds.b[buf]);
            da.load(k, A.ld, lds.a[buf]);
        };
        // A last, partial step goes first, through registers, while the first
        // whole one is on its way to the other buffer.
        if (whole < k1) {
            buf ^= 1;
            if (whole > k0) next(k0);
            buf ^= 1;
            steps(std::true_type{}, whole, k1);
        } else {
            next(k0);
        }
        for (int64_t k = k0; k < whole; k += BK) {
            done();
            __syncthreads();
            buf ^= 1;
            if (k + BK < whole) next(k + BK);
            buf ^= 1;
            compute();
            __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
#pragma unroll
            for (int g = 0; g < kReads; ++g) {
                __builtin_amdgcn_sched_group_barrier(0x008, kProducts / kReads > 0 ? kProducts / kReads : 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, 2 * kProducts, 0);
            buf ^= 1;
        }
    } else {
        if (whole > k0) steps(std::false_type{}, k0, whole);
        if (whole < k1) {
            if (whole > k0) __syncthreads();
            steps(std::true_type{}, whole, k1);
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

// Where tile i of `size` rows starts among `rows`: the last one is moved back
// until it ends with them, as long as there are enough, and then writes its
// rows from `own` on only.  So edges are left to operands smaller than a tile.
struct Span {
    int64_t at, own;
};
__device__ __forceinline__ Span span_of(int64_t i, int64_t size, int64_t rows)
{
    const int64_t own = i * size;
    return Span{max((int64_t)0, min(own, rows - size)), own};
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
