// layer_narrow.h -- linear layers between narrow rows (features of a Gaussian
// to its attributes), of any number of rows: the weights stay in registers and
// the rows stream by, so that memory alone counts.
//
// A wave takes 16 rows at a time (32 in the 16-bit backward pass) straight from
// memory in the layout of the matrix instruction (lane: row l % 16, 16 bytes of
// it at k = 16 bytes x (l / 16)), with the next rows on their way meanwhile.
//   forward:  out = act(x w^T + bias) + residual, or act(g) u with both halves of
//             w in registers; one read of x, one write of out.
//   backward: dz is formed from dout and pre as they are read; it is an operand
//             of dx = dz w as it stands, and passes through a piece of LDS of the
//             wave's own, as x does, to be read down its columns for dw = dz^T x
//             and summed for dbias.  So dout, pre and x are read once, dx is
//             written once, dz never.  The waves' sums of dw and dbias are added
//             up in the block, and the blocks' by a second launch, in order.
// f32 uses the f32 matrix instruction (exact products; at these widths its rate
// is above what memory feeds it).
//
// 1M rows, f32: 32 -> 48 forward 86 us (3.7 TB/s), 32 -> 64 relu backward 166
// (4.6 TB/s; 670 with dz in memory and tiles); 64 -> 64 forward 118, with a
// bias 153, with silu too 170, where the f32 products take 52 and hide only in part.
#pragma once

#include "layer_mm.h"

namespace gsm {

// N values of f32 or S, as f32
template <typename S, int N>
__device__ __forceinline__ void load_f32(const void* p, int64_t at, int type, int64_t valid, float (&v)[N])
{
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        const int n = (int)min((int64_t)4, valid - j);
        const f32x4 x = n > 0 ? load4<S>(p, at + j, type, n) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 4; ++q) v[j + q] = x[q];
    }
}

constexpr int kNarrowThreads = 256;

template <typename S, int KS, int NI, bool GATED>
__global__ __launch_bounds__(kNarrowThreads) void k_narrow_fwd(const LayerMm g)
{
    constexpr int N = 16 / sizeof(S), kStep = 4 * N, kCols = NI * 16, kRow = kCols + 4;
    // A 16-bit result of four columns is 8 bytes: those go through LDS, so that
    // neighbouring lanes write neighbouring columns (64 -> 64 bf16, 1M rows: 123 -> 65 us).
    constexpr bool kTurn = sizeof(S) == 2 && !GATED;
    constexpr int G = GATED ? 2 : 1;
    __shared__ __align__(16) float lds[kTurn ? kNarrowThreads / 64 : 1][kTurn ? 16 * kRow : 4];
    const int lane = threadIdx.x & 63, k0 = (lane >> 4) * N;
    float* const mine = lds[kTurn ? threadIdx.x >> 6 : 0];
    gst::Pack<S, N> b[G][NI][KS];
#pragma unroll
    for (int q = 0; q < G; ++q)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const S* w = (const S*)g.b.p + (q * g.e.n + min((int64_t)(i * 16 + (lane & 15)), g.e.n - 1)) * g.b.ld;
#pragma unroll
            for (int s = 0; s < KS; ++s) b[q][i][s] = upto<S, N>(w + s * kStep + k0, g.k - s * kStep - k0);
        }
    const int64_t groups = (g.m + 15) / 16, stride = (int64_t)gridDim.x * (kNarrowThreads / 64);
    int64_t at = (int64_t)blockIdx.x * (kNarrowThreads / 64) + (threadIdx.x >> 6);
    gst::Pack<S, N> a[KS], next[KS];
    auto load = [&](int64_t group, gst::Pack<S, N>(&v)[KS]) {
        const S* x = (const S*)g.a.p + min(group * 16 + (lane & 15), g.m - 1) * g.a.ld;
#pragma unroll
        for (int s = 0; s < KS; ++s) v[s] = upto<S, N>(x + s * kStep + k0, g.k - s * kStep - k0);
    };
    if (at < groups) load(at, a);
    for (; at < groups; at += stride) {
        if (at + stride < groups) load(at + stride, next);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            f32x4 acc[G];
#pragma unroll
            for (int q = 0; q < G; ++q) {
                acc[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < KS; ++s) acc[q] = mfma16(b[q][i][s], a[s], acc[q]);
            }
            const int row = lane & 15, c = i * 16 + (lane >> 4) * 4;
            const bool there = at * 16 + row < g.m && c < g.e.n;
            if constexpr (kTurn) *reinterpret_cast<f32x4*>(mine + row * kRow + c) = acc[0];
            else if constexpr (GATED) { if (there) epilogue_gated<S>(g.e, at * 16 + row, c, acc[0], acc[1]); }
            else if (there) epilogue<S>(g.e, at * 16 + row, c, acc[0]);
        }
        if constexpr (kTurn) {
            wave_fence();
#pragma unroll
            for (int t = 0; t < NI; ++t) {
                const int q = t * 64 + lane, row = q / (kCols / 4), c = q % (kCols / 4) * 4;
                if (at * 16 + row < g.m && c < g.e.n)
                    epilogue<S>(g.e, at * 16 + row, c, *reinterpret_cast<const f32x4*>(mine + row * kRow + c));
            }
            wave_fence();
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) a[s] = next[s];
    }
}

// What the backward pass of a narrow layer reads and writes; f values of dz and
// k of x a row.
struct NarrowBwd {
    const void *x, *w, *pre, *dout;
    void* dx;                       // null: not wanted
    float* sums;                    // [blocks][f k + f]: dw, then dbias; null: neither is wanted
    int64_t ldx, ldw, ldpre, lddout, lddx;
    int64_t m;
    int32_t f, k, act, dout_type;
};

template <typename S, int FI, int KI>
struct NarrowSize {
    static constexpr int N = 16 / sizeof(S), kStep = 4 * N;          // values of a lane; of a step along a row
    static constexpr int kRows = sizeof(S) == 4 ? 16 : 32;           // of an iteration
    static constexpr int FS = (FI * 16 + kStep - 1) / kStep, XS = (KI * 16 + kStep - 1) / kStep;
    // rows of LDS: columns of 16 neighbouring rows are read at once (f32: 4
    // rows x 16 columns, which 16 words modulo 64 keep apart)
    static constexpr int pad(int cols) { return sizeof(S) == 4 ? cols + (80 - cols % 64) % 64 : cols + 8; }
    static constexpr int ldz = pad(FS * kStep), ldx = pad(XS * kStep);
};

// A wave's rows on their way
template <typename S, int FI, int KI>
struct NarrowRows {
    typedef NarrowSize<S, FI, KI> Z;
    float d[Z::kRows / 16][Z::FS][Z::N];
    gst::Pack<S, Z::N> z[Z::kRows / 16][Z::FS], x[Z::kRows / 16][Z::XS];

    __device__ __forceinline__ void load(const NarrowBwd& g, int64_t row0, int lane)
    {
        const int at = (lane >> 4) * Z::N;
#pragma unroll
        for (int h = 0; h < Z::kRows / 16; ++h) {
            const int64_t m = row0 + h * 16 + (lane & 15);
            const bool there = m < g.m;
            const int64_t r = there ? m : g.m - 1;
#pragma unroll
            for (int s = 0; s < Z::FS; ++s) {
                const int c = s * Z::kStep + at;
                load_f32<S, Z::N>(g.dout, r * g.lddout + c, g.dout_type, there ? g.f - c : 0, d[h][s]);
                if (g.act != GS_ACT_NONE)
                    z[h][s] = upto<S, Z::N>((const S*)g.pre + r * g.ldpre + c, there ? g.f - c : 0);
            }
            if (g.sums) {
#pragma unroll
                for (int s = 0; s < Z::XS; ++s) {
                    const int c = s * Z::kStep + at;
                    x[h][s] = upto<S, Z::N>((const S*)g.x + r * g.ldx + c, there ? g.k - c : 0);
                }
            }
        }
    }
};

// acc += 16 columns of x (from cx on) and of dz (from cz on) over a wave's rows
template <typename S, typename Z>
__device__ __forceinline__ f32x4 column_product(const S* x, int cx, const S* z, int cz, int lane, f32x4 acc)
{
    if constexpr (sizeof(S) == 4) {
#pragma unroll
        for (int q = 0; q < Z::kRows / 4; ++q) {
            const int r = q * 4 + (lane >> 4);
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r * Z::ldx + cx + (lane & 15)], z[r * Z::ldz + cz + (lane & 15)],
                                                       acc, 0, 0, 0);
        }
        return acc;
    } else {
        auto part = [&](const S* p, int ld, int c) {
            typedef short v4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) v4* at;
            const S* q = p + ((lane >> 4) * 8 + ((lane >> 2) & 3)) * ld + c + (lane & 3) * 4;
            const v4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at)q);
            const v4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at)(q + 4 * ld));
            gst::Pack<S, 8> both;
            __builtin_memcpy(&both.v[0], &lo, 8);
            __builtin_memcpy(&both.v[4], &hi, 8);
            return both;
        };
        return mfma(part(x, Z::ldx, cx), part(z, Z::ldz, cz), acc);
    }
}

template <typename S, int FI, int KI>
__global__ __launch_bounds__(kNarrowThreads, 2) void k_narrow_bwd(const NarrowBwd g)
{
    typedef NarrowSize<S, FI, KI> Z;
    constexpr int W = kNarrowThreads / 64, N = Z::N;
    constexpr bool kScaled = std::is_same<S, gst::f16>::value;   // dz as in k_dz: by a row's scale for dx, by a wave's for dw
    // The next rows are on their way while these are worked on, where registers
    // for both leave two waves a SIMD (1M x 32 -> 64 f32: 167 us, 182 without;
    // 64 -> 64 f32: 425, 270 without; the 16-bit types lose at every width).
    constexpr bool PRE = sizeof(S) == 4 && FI * KI <= 9;
    __shared__ __align__(16) union {
        S rows[W][Z::kRows * (Z::ldz + Z::ldx)];
        float sums[FI * KI * 256 + FI * 16];
    } lds;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, at = (lane >> 4) * N;
    gst::Pack<S, N> w[KI][Z::FS];   // w^T as an operand: row k, values of f
    if (g.dx) {
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int k = min(i * 16 + (lane & 15), g.k - 1);
#pragma unroll
            for (int s = 0; s < Z::FS; ++s)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int f = s * Z::kStep + at + j;
                    w[i][s].v[j] = f < g.f ? ((const S*)g.w)[(int64_t)f * g.ldw + k] : (S)0.0f;
                }
        }
    }
    f32x4 dw[FI][KI];
#pragma unroll
    for (int f = 0; f < FI; ++f)
#pragma unroll
        for (int k = 0; k < KI; ++k) dw[f][k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    int scale = 126;   // f16: exponent by which dz is scaled in dw's sums
    float db[Z::FS][N];
#pragma unroll
    for (int s = 0; s < Z::FS; ++s)
#pragma unroll
        for (int j = 0; j < N; ++j) db[s][j] = 0.0f;
    S* const lz = lds.rows[wave];
    S* const lx = lz + Z::kRows * Z::ldz;
    const int64_t stride = (int64_t)gridDim.x * W * Z::kRows;
    int64_t row0 = ((int64_t)blockIdx.x * W + wave) * Z::kRows;
    NarrowRows<S, FI, KI> now, next;
    if (PRE && row0 < g.m) now.load(g, row0, lane);
    for (; row0 < g.m; row0 += stride) {
        if constexpr (PRE) {
            if (row0 + stride < g.m) next.load(g, row0 + stride, lane);
        } else {
            now.load(g, row0, lane);
        }
        // dz, in place of dout; f16: all of it before the first is rounded
        float most[Z::kRows / 16];
        auto form = [&](int h) {
            most[h] = 0.0f;
#pragma unroll
            for (int s = 0; s < Z::FS; ++s)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    float& v = now.d[h][s][j];
                    if (g.act != GS_ACT_NONE) v *= act_both((float)now.z[h][s].v[j], g.act).y;
                    // past the last value of a row, and past the last row, pre is 0 and dout too
                    db[s][j] += v;
                    if constexpr (kScaled) most[h] = larger(most[h], v);
                }
        };
        if constexpr (kScaled) {
            // each row's largest, and the rows' together; sums so far follow when theirs is the largest yet
            float all = 0.0f;
#pragma unroll
            for (int h = 0; h < Z::kRows / 16; ++h) {
                form(h);
                most[h] = fmaxf(most[h], __shfl_xor(most[h], 16));
                most[h] = fmaxf(most[h], __shfl_xor(most[h], 32));
                all = fmaxf(all, most[h]);
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) all = fmaxf(all, __shfl_xor(all, d));
            const int e = __builtin_amdgcn_readfirstlane(all > 0.0f ? scale_exponent(all) : 126);
            if (e < scale) {
#pragma unroll
                for (int f = 0; f < FI; ++f)
#pragma unroll
                    for (int k = 0; k < KI; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j) dw[f][k][j] = ldexpf(dw[f][k][j], e - scale);
                scale = e;
            }
        }
#pragma unroll
        for (int h = 0; h < Z::kRows / 16; ++h) {
            if constexpr (!kScaled) form(h);
            const int by_row = kScaled ? scale_exponent(most[h]) : 0;
            gst::Pack<S, N> dz[Z::FS];
            auto round = [&](int e) {
#pragma unroll
                for (int s = 0; s < Z::FS; ++s)
#pragma unroll
                    for (int j = 0; j < N; ++j) dz[s].v[j] = gst::narrow<S>(kScaled ? ldexpf(now.d[h][s][j], e) : now.d[h][s][j]);
            };
            round(by_row);
            if (g.dx) {
                const int64_t m = row0 + h * 16 + (lane & 15);
#pragma unroll
                for (int i = 0; i < KI; ++i) {
                    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < Z::FS; ++s) acc = mfma16(w[i][s], dz[s], acc);
                    if constexpr (kScaled) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[j] = ldexpf(acc[j], -by_row);
                    }
                    const int c = i * 16 + (lane >> 4) * 4;
                    if (m < g.m && c < g.k) store4<S>(g.dx, m * g.lddx + c, sizeof(S) == 4 ? GS_F32 : -1, g.k - c, acc);
                }
            }
            if (g.sums) {
                if constexpr (kScaled) round(scale);
                const int r = h * 16 + (lane & 15);
#pragma unroll
                for (int s = 0; s < Z::FS; ++s)
                    *reinterpret_cast<gst::Pack<S, N>*>(__builtin_assume_aligned(lz + r * Z::ldz + s * Z::kStep + at, 16)) = dz[s];
#pragma unroll
                for (int s = 0; s < Z::XS; ++s)
                    *reinterpret_cast<gst::Pack<S, N>*>(__builtin_assume_aligned(lx + r * Z::ldx + s * Z::kStep + at, 16)) =
                        now.x[h][s];
            }
        }
        if (g.sums) {
            wave_fence();
#pragma unroll
            for (int f = 0; f < FI; ++f)
#pragma unroll
                for (int k = 0; k < KI; ++k) dw[f][k] = column_product<S, Z>(lx, k * 16, lz, f * 16, lane, dw[f][k]);
            wave_fence();
        }
        if constexpr (PRE) now = next;
    }
    if (!g.sums) return;
    if constexpr (kScaled) {
#pragma unroll
        for (int f = 0; f < FI; ++f)
#pragma unroll
            for (int k = 0; k < KI; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) dw[f][k][j] = ldexpf(dw[f][k][j], -scale);
    }
    // the block's sums, wave after wave
#pragma unroll
    for (int s = 0; s < Z::FS; ++s)
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) db[s][j] += __shfl_xor(db[s][j], d);
    for (int v = 0; v < W; ++v) {
        __syncthreads();
        if (wave != v) continue;
#pragma unroll
        for (int f = 0; f < FI; ++f)
#pragma unroll
            for (int k = 0; k < KI; ++k) {
                f32x4* to = reinterpret_cast<f32x4*>(lds.sums + (f * KI + k) * 256 + lane * 4);
                *to = v ? *to + dw[f][k] : dw[f][k];
            }
        if ((lane & 15) == 0) {
#pragma unroll
            for (int s = 0; s < Z::FS; ++s)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int f = s * Z::kStep + at + j;
                    if (f < FI * 16) lds.sums[FI * KI * 256 + f] = db[s][j] + (v ? lds.sums[FI * KI * 256 + f] : 0.0f);
                }
        }
    }
    __syncthreads();
    float* out = g.sums + (int64_t)blockIdx.x * ((int64_t)g.f * g.k + g.f);
    for (int t = threadIdx.x; t < g.f * g.k + g.f; t += kNarrowThreads) {
        int from = FI * KI * 256 + t - g.f * g.k;
        if (t < g.f * g.k) {
            const int f = t / g.k, k = t % g.k;   // of the lane's place: f its l % 16, k its 4 (l / 16) + 0..3
            from = ((f >> 4) * KI + (k >> 4)) * 256 + (((k & 15) >> 2) * 16 + (f & 15)) * 4 + (k & 3);
        }
        out[t] = lds.sums[from];
    }
}

// the widths that have kernels, in blocks of 16: f(constants) for the least that hold them
template <int MOST, typename F>
bool with_blocks(int64_t a, int64_t b, F&& f)
{
    auto second = [&](auto i) {
        constexpr int A = decltype(i)::value;
        if constexpr (A * 1 <= MOST) { if (b <= 1) { f(i, std::integral_constant<int, 1>{}); return true; } }
        if constexpr (A * 2 <= MOST) { if (b <= 2) { f(i, std::integral_constant<int, 2>{}); return true; } }
        if constexpr (A * 3 <= MOST) { if (b <= 3) { f(i, std::integral_constant<int, 3>{}); return true; } }
        if constexpr (A * 4 <= MOST) { if (b <= 4) { f(i, std::integral_constant<int, 4>{}); return true; } }
        if constexpr (A * 8 <= MOST) { if (b <= 8) { f(i, std::integral_constant<int, 8>{}); return true; } }
        return false;
    };
    if (a <= 1) return second(std::integral_constant<int, 1>{});
    if (a <= 2) return second(std::integral_constant<int, 2>{});
    if (a <= 3) return second(std::integral_constant<int, 3>{});
    if (a <= 4) return second(std::integral_constant<int, 4>{});
    if (a <= 8) return second(std::integral_constant<int, 8>{});
    return false;
}

constexpr int kNarrowFwd = 24, kNarrowBwd = 16;   // operands of w, and results of dw, that a wave holds in registers

// Blocks of the backward pass: two a compute unit, four for the least widths
// (1M rows of 32 -> 3 f32: 73 us, 95 with two; of 64 -> 64: 270 with two, 292).
inline int64_t narrow_blocks(const gs_ctx* ctx, int type, int64_t m, int64_t f, int64_t k)
{
    const int64_t rows = (type == GS_F32 ? 16 : 32) * (kNarrowThreads / 64);
    return std::min(ceil_div(m, rows), (ceil_div(f, 16) * ceil_div(k, 16) <= 2 ? 4 : 2) * (int64_t)ctx->num_cu);
}

// blocks of w that a wave holds: pieces of a row as the matrix instruction takes them, and of 16 columns
template <typename S>
inline int64_t narrow_steps(int64_t k)
{
    return ceil_div(k, 64 / (int64_t)sizeof(S));
}
// whether the forward pass has a kernel
inline bool narrow_fwd(int type, const LayerMm& g)
{
    const int64_t steps = type == GS_F32 ? narrow_steps<float>(g.k) : narrow_steps<gst::f16>(g.k), cols = ceil_div(g.e.n, 16);
    return g.gated ? with_blocks<kNarrowFwd / 2>(steps, cols, [](auto, auto) {})
                   : with_blocks<kNarrowFwd>(steps, cols, [](auto, auto) {});
}
// whether the backward pass of f x k weights has a kernel
inline bool narrow_bwd(int64_t f, int64_t k)
{
    return with_blocks<kNarrowBwd>(ceil_div(f, 16), ceil_div(k, 16), [](auto, auto) {});
}

// one type each (layer_narrow_*.hip), for widths that narrow_fwd or narrow_bwd allow
void launch_narrow_fwd_f32(gs_ctx* ctx, const LayerMm& g);
void launch_narrow_fwd_f16(gs_ctx* ctx, const LayerMm& g);
void launch_narrow_fwd_bf16(gs_ctx* ctx, const LayerMm& g);
void launch_narrow_bwd_f32(gs_ctx* ctx, const NarrowBwd& g, int64_t blocks);
void launch_narrow_bwd_f16(gs_ctx* ctx, const NarrowBwd& g, int64_t blocks);
void launch_narrow_bwd_bf16(gs_ctx* ctx, const NarrowBwd& g, int64_t blocks);

template <typename S, bool GATED>
void launch_narrow_rows(gs_ctx* ctx, const LayerMm& g)
{
    with_blocks<kNarrowFwd / (GATED ? 2 : 1)>(narrow_steps<S>(g.k), ceil_div(g.e.n, 16), [&](auto ks, auto ni) {
        // waves that come back for more rows: 6 blocks a compute unit, and where
        // w takes few registers 24 (32 -> 48 f32: 86 us, 106 with 6; 64 -> 64: 184, 170)
        constexpr int kOps = decltype(ks)::value * decltype(ni)::value * (GATED ? 2 : 1);
        const int64_t groups = ceil_div(g.m, 16 * (kNarrowThreads / 64)),
                      most = (sizeof(S) == 2 || kOps > 8 ? 6 : 24) * ctx->num_cu;
        hipLaunchKernelGGL((k_narrow_fwd<S, decltype(ks)::value, decltype(ni)::value, GATED>),
                           dim3((uint32_t)std::min(groups, most)), dim3(kNarrowThreads), 0, ctx->stream, g);
    });
}

template <typename S>
void launch_narrow_fwd(gs_ctx* ctx, const LayerMm& g)
{
    if (g.gated) launch_narrow_rows<S, true>(ctx, g);
    else launch_narrow_rows<S, false>(ctx, g);
}

template <typename S>
void launch_narrow_bwd(gs_ctx* ctx, const NarrowBwd& g, int64_t blocks)
{
    with_blocks<kNarrowBwd>(ceil_div(g.f, 16), ceil_div(g.k, 16), [&](auto fi, auto ki) {
        hipLaunchKernelGGL((k_narrow_bwd<S, decltype(fi)::value, decltype(ki)::value>), dim3((uint32_t)blocks),
                           dim3(kNarrowThreads), 0, ctx->stream, g);
    });
}

}  // namespace gsm
