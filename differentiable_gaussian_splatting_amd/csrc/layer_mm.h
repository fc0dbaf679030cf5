// layer_mm.h -- the matrix products of linear and gated layers: the kernel
// over tiles with its epilogues, and the launch for one element type (the
// layer_mm_*.hip files instantiate one each).
//
//   linear: out = act(x w^T + bias) + residual
//   gated:  [g u] = x w^T, out = act(g) u
//   gradients: dx = dz w, dw = dz^T x
//
// A lane holds four neighbouring columns of one row, so the epilogue reads
// bias and residual and writes its outputs in packs of four.  Everything in it
// is f32; each output is rounded once.
//
// Large products are bound by the matrix cores: 8192^3 bf16 970 to 990 us, 1110
// to 1130 TFLOP/s (the library's product 1530 to 1570 on the same cards); 8192 x
// 4096 -> 2 x 11008 gated bf16 1490 to 1560 (950 to 990 TFLOP/s), where 540 MB of
// outputs are written after the products of a tile; f32 in three parts 8192 x
// 2048 -> 4096 680 to 790 us (175 to 200 TFLOP/s, 1050 to 1200 of the 16-bit
// products; the library's f32 product 148).
#pragma once

#include <algorithm>

#include "gs_internal.h"
#include "layers.h"
#include "mm.h"

namespace gsm {

typedef gst::Pack<float, 4> Four;

// Values [first, valid) of the four from p[at] on.
template <typename S>
__device__ __forceinline__ f32x4 load4(const void* p, int64_t at, int type, int valid, int first = 0)
{
    f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
    if (type == GS_F32) {
        const float* q = (const float*)p + at;
        if (valid >= 4 && first == 0) return __builtin_bit_cast(f32x4, gst::load<float, 4>(q));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j >= first && j < valid) r[j] = q[j];
    } else {
        const S* q = (const S*)p + at;
        if (valid >= 4 && first == 0) {
            const gst::Pack<S, 4> v = gst::load<S, 4>(q);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = (float)v.v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j >= first && j < valid) r[j] = (float)q[j];
        }
    }
    return r;
}

template <typename S>
__device__ __forceinline__ void store4(void* p, int64_t at, int type, int valid, f32x4 x, int first = 0)
{
    if (type == GS_F32) {
        float* q = (float*)p + at;
        if (valid >= 4 && first == 0) {
            gst::store<float, 4>(q, __builtin_bit_cast(Four, x));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j >= first && j < valid) q[j] = x[j];
        }
    } else {
        S* q = (S*)p + at;
        gst::Pack<S, 4> v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v.v[j] = gst::narrow<S>(x[j]);
        if (valid >= 4 && first == 0) {
            gst::store<S, 4>(q, v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j >= first && j < valid) q[j] = v.v[j];
        }
    }
}

// 16 x 16 results from 16 bytes of k per lane
__device__ __forceinline__ f32x4 mfma16(gst::Pack<float, 4> a, gst::Pack<float, 4> b, f32x4 c)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
    return c;
}
template <typename E>
__device__ __forceinline__ f32x4 mfma16(gst::Pack<E, 8> a, gst::Pack<E, 8> b, f32x4 c)
{
    return mfma(a, b, c);
}

// N values from p on, zeros from the n-th one on (n may be negative)
template <typename S, int N>
__device__ __forceinline__ gst::Pack<S, N> upto(const S* p, int64_t n)
{
    if (n >= N) return gst::load<S, N>(p);
    gst::Pack<S, N> v;
#pragma unroll
    for (int j = 0; j < N; ++j) v.v[j] = j < n ? p[j] : (S)0.0f;
    return v;
}

// columns n + first .. n + 3 of row m of the product; DOWN: e.down may be there
template <typename S, bool DOWN = false>
__device__ __forceinline__ void epilogue(const Epilogue& e, int64_t m, int64_t n, f32x4 z, int first = 0)
{
    const int valid = (int)min((int64_t)4, e.n - n);
    if constexpr (DOWN) { if (e.down) z *= e.down[m * e.lddown]; }
    if (e.bias) z += load4<S>(e.bias, n, e.bias_type, valid, first);
    if (e.pre) store4<S>(e.pre, m * e.ldpre + n, e.pre_type, valid, z, first);
    if (e.act != GS_ACT_NONE) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = act_value(z[j], e.act);
    }
    if (e.res) z += load4<S>(e.res, m * e.ldres + n, e.res_type, valid, first);
    store4<S>(e.out, m * e.ldout + n, e.out_type, valid, z, first);
}

// columns f + first .. f + 3 of row m of both halves
template <typename S>
__device__ __forceinline__ void epilogue_gated(const Epilogue& e, int64_t m, int64_t f, f32x4 g, f32x4 u, int first = 0)
{
    const int valid = (int)min((int64_t)4, e.n - f);
    if (e.pre) {
        store4<S>(e.pre, m * e.ldpre + f, e.pre_type, valid, g, first);
        store4<S>(e.pre, m * e.ldpre + e.n + f, e.pre_type, valid, u, first);
    }
    f32x4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = act_value(g[j], e.act) * u[j];
    store4<S>(e.out, m * e.ldout + f, e.out_type, valid, y, first);
}

// A wave's LDS writes are there for its own reads.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// f32 in parts: an infinity, or a value above bf16's largest, has parts whose
// products meet as NaN.  So where a result is NaN the products of its values
// themselves are summed, which ends at the first NaN: the four of row m from
// column n on, b's rows from `row` on.
template <bool ACOL, bool BCOL>
__device__ __forceinline__ f32x4 sum_again(const Operand& a, const Operand& b, int64_t m, int64_t row, int valid, int64_t k0,
                                           int64_t k1, f32x4 z)
{
    const float any = (z[0] + z[1]) + (z[2] + z[3]);
    if (any == any) return z;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        if (z[j] == z[j] || j >= valid) continue;
        const float* x = (const float*)a.p + (ACOL ? k0 * a.ld + m : m * a.ld + k0);
        const float* w = (const float*)b.p + (BCOL ? k0 * b.ld + row + j : (row + j) * b.ld + k0);
        float s = 0.0f;
        for (int64_t k = k0; k < k1 && s == s; ++k) {
            s = fmaf(*x, *w, s);
            x += ACOL ? a.ld : 1;
            w += BCOL ? b.ld : 1;
        }
        z[j] = s;
    }
    return z;
}

// Tiles of the product (DIRECT: see mm_tile); those from `full` on in `splits` ranges of k, whose sums
// k_join adds up.
template <typename S, int P, typename T>
union LayerLds {
    Lds<S, P, T> tile;
    float out[T::NT / 64 * 32 * (T::NI * 16 + 4)];
};

// block `block` of `blocks` that form the product
template <typename S, int P, bool ACOL, bool BCOL, bool GATED, typename T, bool DIRECT>
__device__ __forceinline__ void layer_mm(const LayerMm& g, int64_t block, int64_t blocks, LayerLds<S, P, T>& lds)
{
    constexpr int kCols = T::NI * (GATED ? 8 : 16), kRow = T::NI * 16 + 4;   // of a wave's results; padded row in LDS
    constexpr int G = GATED ? 2 : 1;
    const int64_t rest = g.tm * g.tn - g.full, total = g.full + rest * g.splits;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // only the gradients' products have a scaled dz; the code of the others stays without it
    // (8192 x 4096 -> 11008 bf16 forward 880 us with it, 843 without)
    constexpr bool kScaled = std::is_same<S, f16>::value && BCOL;
    Operand ga = g.a;
    if constexpr (kScaled) { if (g.other && *g.other) ga.p = g.a_other; }
    for (int64_t b = block; b < total; b += blocks) {
        int64_t tile = b, k0 = 0, k1 = g.k, i, j;
        float* ws = nullptr;
        if (b < g.full) {
            tile = xcd_order(b, g.full);
        } else {
            const int64_t at = xcd_order(b - g.full, rest * g.splits), s = at / rest;
            tile = g.full + at % rest;
            k0 = s * g.kper;
            k1 = min(g.k, k0 + g.kper);
            ws = g.ws + at * (T::BM * T::BN);
        }
        tile_at(tile, g.tm, g.tn, i, j);
        const Span sm = span_of(i, T::BM, g.a.rows), sn = span_of(j, T::BN / G, GATED ? g.e.n : g.b.rows);
        const int64_t m0 = sm.at, n0 = sn.at * G;
        f32x4 acc[T::NI][T::MI];
#pragma unroll
        for (int q = 0; q < T::NI; ++q)
#pragma unroll
            for (int r = 0; r < T::MI; ++r) acc[q][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (b != block) __syncthreads();   // the previous tile's reads of lds
        mm_tile<S, P, ACOL, BCOL, T, false, DIRECT>(kScaled ? ga : g.a, g.b, m0, n0, k0, k1, lds.tile, acc);
        // The results go through LDS, 32 rows of each wave at a time, so that a
        // lane takes four columns next to its neighbours' (whole lines are
        // read and written) and the epilogue's code is a loop.
        __syncthreads();
        float* mine = reinterpret_cast<float*>(&lds) + wave * 32 * kRow;
        const int64_t mw = m0 + (wave % T::WM) * T::MI * 16;
        const int64_t nw = sn.at + (wave / T::WM) * kCols;
#pragma unroll
        for (int r = 0; r < T::MI; r += 2) {
            if (mw + r * 16 >= g.m) break;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < T::NI; ++q)
                    *reinterpret_cast<f32x4*>(mine + (h * 16 + (lane & 15)) * kRow + q * 16 + (lane >> 4) * 4) = acc[q][r + h];
            wave_fence();
            for (int t = lane; t < 32 * kCols / 4; t += 64) {
                const int row = t / (kCols / 4), c = t % (kCols / 4) * 4;
                const int64_t m = mw + r * 16 + row, n = nw + c;
                if (m >= g.m || n >= g.e.n || m < sm.own || n + 3 < sn.own) continue;
                const int first = (int)max((int64_t)0, sn.own - n);
                const float* v = mine + row * kRow + (GATED ? (c >> 4) * 32 + (c & 15) : c);
                f32x4 x = *reinterpret_cast<const f32x4*>(v), y;
                if constexpr (P == 3) x = sum_again<ACOL, BCOL>(g.a, g.b, m, n, (int)min((int64_t)4, g.e.n - n), k0, k1, x);
                if constexpr (GATED && P == 3)
                    y = sum_again<ACOL, BCOL>(g.a, g.b, m, g.e.n + n, (int)min((int64_t)4, g.e.n - n), k0, k1,
                                              *reinterpret_cast<const f32x4*>(v + 16));
                if (ws) {
                    float* w = ws + (m - m0) * T::BN + (wave / T::WM) * T::NI * 16 + (v - mine - row * kRow);
                    *reinterpret_cast<f32x4*>(w) = x;
                    if constexpr (GATED) *reinterpret_cast<f32x4*>(w + 16) = P == 3 ? y : *reinterpret_cast<const f32x4*>(v + 16);
                } else if constexpr (GATED) {
                    epilogue_gated<S>(g.e, m, n, x, P == 3 ? y : *reinterpret_cast<const f32x4*>(v + 16), first);
                } else {
                    epilogue<S, kScaled>(g.e, m, n, x, first);
                }
            }
            wave_fence();
        }
    }
}

template <typename S, int P, bool ACOL, bool BCOL, bool GATED, typename T, bool DIRECT>
__global__ __launch_bounds__(T::NT, 2) void k_layer_mm(const LayerMm g)
{
    __shared__ LayerLds<S, P, T> lds;
    layer_mm<S, P, ACOL, BCOL, GATED, T, DIRECT>(g, blockIdx.x, gridDim.x, lds);
}

// dx and dw of a small layer in one launch: the first `split` blocks form dx
template <typename S, int P, typename T>
__global__ __launch_bounds__(T::NT, 2) void k_layer_pair(const LayerMm x, const LayerMm w, int split)
{
    __shared__ LayerLds<S, P, T> lds;
    if ((int)blockIdx.x < split) layer_mm<S, P, false, true, false, T, false>(x, blockIdx.x, split, lds);
    else layer_mm<S, P, true, true, false, T, false>(w, blockIdx.x - split, gridDim.x - split, lds);
}

// Sums of the splits in their order, then the epilogue; four columns a thread.
template <typename S, bool GATED, typename T>
__global__ __launch_bounds__(256) void k_join(const LayerMm g)
{
    constexpr int kCols = T::BN / (GATED ? 2 : 1), kQuads = T::BM * kCols / 4;
    const int64_t rest = g.tm * g.tn - g.full, total = rest * kQuads;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t tile = t / kQuads;
        const int row = t % kQuads / (kCols / 4), c = t % (kCols / 4) * 4;
        int64_t i, j;
        tile_at(g.full + tile, g.tm, g.tn, i, j);
        const Span sm = span_of(i, T::BM, g.a.rows), sn = span_of(j, kCols, GATED ? g.e.n : g.b.rows);
        const int64_t m = sm.at + row, n = sn.at + c;
        if (m >= g.m || n >= g.e.n || m < sm.own || n + 3 < sn.own) continue;
        const float* w = g.ws + tile * (T::BM * T::BN) + row * T::BN + (GATED ? (c >> 4) * 32 + (c & 15) : c);
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll 4
        for (int s = 0; s < g.splits; ++s) {
            x += *reinterpret_cast<const f32x4*>(w + s * rest * (T::BM * T::BN));
            if constexpr (GATED) y += *reinterpret_cast<const f32x4*>(w + s * rest * (T::BM * T::BN) + 16);
        }
        const int first = (int)max((int64_t)0, sn.own - n);
        if constexpr (GATED) epilogue_gated<S>(g.e, m, n, x, y, first);
        else epilogue<S, std::is_same<S, f16>::value>(g.e, m, n, x, first);
    }
}

constexpr int64_t kMaxGrid = 1 << 22;   // blocks of a launch; larger products loop

inline int64_t layer_blocks(const LayerMm& g)
{
    return std::min(g.full + (g.tm * g.tn - g.full) * g.splits, kMaxGrid);
}

template <typename S, typename T>
void launch_join(gs_ctx* ctx, const LayerMm& g)
{
    if (g.splits == 1) return;
    const int64_t quads = (g.tm * g.tn - g.full) * T::BM * T::BN / (g.gated ? 8 : 4);
    const dim3 grid((uint32_t)std::min(ceil_div(quads, 256), kMaxGrid));
    if (g.gated) hipLaunchKernelGGL((k_join<S, true, T>), grid, dim3(256), 0, ctx->stream, g);
    else hipLaunchKernelGGL((k_join<S, false, T>), grid, dim3(256), 0, ctx->stream, g);
}

template <typename S, int P, typename T, bool DIRECT>
void launch_mode(gs_ctx* ctx, const LayerMm& g)
{
    const dim3 grid((uint32_t)layer_blocks(g)), block(T::NT);
    if (g.a_col) hipLaunchKernelGGL((k_layer_mm<S, P, true, true, false, T, DIRECT>), grid, block, 0, ctx->stream, g);
    else if (g.b_col) hipLaunchKernelGGL((k_layer_mm<S, P, false, true, false, T, DIRECT>), grid, block, 0, ctx->stream, g);
    else if (g.gated) hipLaunchKernelGGL((k_layer_mm<S, P, false, false, true, T, DIRECT>), grid, block, 0, ctx->stream, g);
    else hipLaunchKernelGGL((k_layer_mm<S, P, false, false, false, T, DIRECT>), grid, block, 0, ctx->stream, g);
    launch_join<S, T>(ctx, g);
}

template <typename S, int P, typename Large, typename Medium, typename Small, typename Tiny>
gs_status launch_layer_mm(gs_ctx* ctx, const LayerMm& g)
{
    GsTimerScope ts(ctx, "layer_mm");
    const bool direct = P == 1 && loads_direct(g);
    if (g.tile == kLarge && direct) launch_mode<S, P, Large, P == 1>(ctx, g);
    else if (g.tile == kLarge) launch_mode<S, P, Large, false>(ctx, g);
    else if (g.tile == kMedium && direct) launch_mode<S, P, Medium, P == 1>(ctx, g);
    else if (g.tile == kMedium) launch_mode<S, P, Medium, false>(ctx, g);
    else if (g.tile == kSmall) launch_mode<S, P, Small, false>(ctx, g);
    else launch_mode<S, P, Tiny, false>(ctx, g);
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

// dx and dw, both of small tiles
template <typename S, int P, typename Small>
gs_status launch_layer_pair(gs_ctx* ctx, const LayerMm& x, const LayerMm& w)
{
    GsTimerScope ts(ctx, "layer_mm");
    const int64_t split = layer_blocks(x);
    hipLaunchKernelGGL((k_layer_pair<S, P, Small>), dim3((uint32_t)(split + layer_blocks(w))), dim3(Small::NT), 0, ctx->stream,
                       x, w, (int)split);
    launch_join<S, Small>(ctx, x);
    launch_join<S, Small>(ctx, w);
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

}  // namespace gsm
