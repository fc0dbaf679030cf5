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
#pragma once

#include <algorithm>

#include "gs_internal.h"
#include "layers.h"
#include "mm.h"

namespace gsm {

typedef gst::Pack<float, 4> Four;

template <typename S>
__device__ __forceinline__ f32x4 load4(const void* p, int64_t at, int type, int valid)
{
    f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
    if (type == GS_F32) {
        const float* q = (const float*)p + at;
        if (valid >= 4) return __builtin_bit_cast(f32x4, gst::load<float, 4>(q));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < valid) r[j] = q[j];
    } else {
        const S* q = (const S*)p + at;
        if (valid >= 4) {
            const gst::Pack<S, 4> v = gst::load<S, 4>(q);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = (float)v.v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < valid) r[j] = (float)q[j];
        }
    }
    return r;
}

template <typename S>
__device__ __forceinline__ void store4(void* p, int64_t at, int type, int valid, f32x4 x)
{
    if (type == GS_F32) {
        float* q = (float*)p + at;
        if (valid >= 4) {
            gst::store<float, 4>(q, __builtin_bit_cast(Four, x));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < valid) q[j] = x[j];
        }
    } else {
        S* q = (S*)p + at;
        gst::Pack<S, 4> v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v.v[j] = gst::narrow<S>(x[j]);
        if (valid >= 4) {
            gst::store<S, 4>(q, v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < valid) q[j] = v.v[j];
        }
    }
}

// columns n .. n + 3 of row m of the product
template <typename S>
__device__ __forceinline__ void epilogue(const Epilogue& e, int64_t m, int64_t n, f32x4 z)
{
    const int valid = (int)min((int64_t)4, e.n - n);
    if (e.bias) z += load4<S>(e.bias, n, e.bias_type, valid);
    if (e.pre) store4<S>(e.pre, m * e.ldpre + n, e.pre_type, valid, z);
    if (e.act != GS_ACT_NONE) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = act_value(z[j], e.act);
    }
    if (e.res) z += load4<S>(e.res, m * e.ldres + n, e.res_type, valid);
    store4<S>(e.out, m * e.ldout + n, e.out_type, valid, z);
}

// columns f .. f + 3 of row m of both halves
template <typename S>
__device__ __forceinline__ void epilogue_gated(const Epilogue& e, int64_t m, int64_t f, f32x4 g, f32x4 u)
{
    const int valid = (int)min((int64_t)4, e.n - f);
    if (e.pre) {
        store4<S>(e.pre, m * e.ldpre + f, e.pre_type, valid, g);
        store4<S>(e.pre, m * e.ldpre + e.n + f, e.pre_type, valid, u);
    }
    f32x4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = act_value(g[j], e.act) * u[j];
    store4<S>(e.out, m * e.ldout + f, e.out_type, valid, y);
}

// A wave's LDS writes are there for its own reads.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Tiles of the product, each over one of `splits` ranges of k; with more than
// one, the sums go to ws [split][m][wn] and k_join adds them up.
template <typename S, int P, bool ACOL, bool BCOL, bool GATED, typename T>
__global__ __launch_bounds__(T::NT, 2) void k_layer_mm(const LayerMm g)
{
    constexpr int kCols = T::NI * (GATED ? 8 : 16), kRow = T::NI * 16 + 4;   // of a wave's results; padded row in LDS
    __shared__ union {
        Lds<S, P, T> tile;
        float out[T::NT / 64 * 32 * kRow];
    } lds;
    const int64_t tiles = g.tm * g.tn, total = tiles * g.splits;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int64_t at = xcd_order(b, total), s = at / tiles;
        int64_t i, j;
        tile_at(at % tiles, g.tm, g.tn, i, j);
        const int64_t m0 = i * T::BM, n0 = j * T::BN, k0 = s * g.kper;
        f32x4 acc[T::NI][T::MI];
#pragma unroll
        for (int q = 0; q < T::NI; ++q)
#pragma unroll
            for (int r = 0; r < T::MI; ++r) acc[q][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (b != (int64_t)blockIdx.x) __syncthreads();   // the previous tile's reads of lds
        mm_tile<S, P, ACOL, BCOL, T>(g.a, g.b, m0, n0, k0, min(g.k, k0 + g.kper), lds.tile, acc);
        // The results go through LDS, 32 rows of each wave at a time, so that a
        // lane takes four columns next to its neighbours' (whole lines are
        // read and written) and the epilogue's code is a loop.
        __syncthreads();
        float* mine = reinterpret_cast<float*>(&lds) + wave * 32 * kRow;
        const int64_t mw = m0 + (wave % T::WM) * T::MI * 16;
        const int64_t nw = n0 / (GATED ? 2 : 1) + (wave / T::WM) * kCols;
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
                if (m >= g.m || n >= g.e.n) continue;
                const float* v = mine + row * kRow + (GATED ? (c >> 4) * 32 + (c & 15) : c);
                const f32x4 x = *reinterpret_cast<const f32x4*>(v);
                if (g.splits > 1) {
                    float* w = g.ws + (s * g.m + m) * g.wn + n;
                    gst::store<float, 4>(w, __builtin_bit_cast(Four, x));
                    if constexpr (GATED) gst::store<float, 4>(w + g.wn / 2, *reinterpret_cast<const Four*>(v + 16));
                } else if constexpr (GATED) {
                    epilogue_gated<S>(g.e, m, n, x, *reinterpret_cast<const f32x4*>(v + 16));
                } else {
                    epilogue<S>(g.e, m, n, x);
                }
            }
            wave_fence();
        }
    }
}

// Sums of the splits in their order, then the epilogue; four columns a thread.
template <typename S, bool GATED>
__global__ __launch_bounds__(256) void k_join(const LayerMm g)
{
    const int64_t n4 = (g.e.n + 3) / 4, total = g.m * n4;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t m = t / n4, n = t % n4 * 4;
        const float* w = g.ws + m * g.wn + n;
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
        for (int s = 0; s < g.splits; ++s) {
            x += __builtin_bit_cast(f32x4, gst::load<float, 4>(w + s * g.m * g.wn));
            if constexpr (GATED) y += __builtin_bit_cast(f32x4, gst::load<float, 4>(w + s * g.m * g.wn + g.wn / 2));
        }
        if constexpr (GATED) epilogue_gated<S>(g.e, m, n, x, y);
        else epilogue<S>(g.e, m, n, x);
    }
}

constexpr int64_t kMaxGrid = 1 << 22;   // blocks of a launch; larger products loop

template <typename S, int P, typename T>
void launch_mode(gs_ctx* ctx, const LayerMm& g)
{
    const dim3 grid((uint32_t)std::min(g.tm * g.tn * g.splits, kMaxGrid)), block(T::NT);
    if (g.a_col) hipLaunchKernelGGL((k_layer_mm<S, P, true, true, false, T>), grid, block, 0, ctx->stream, g);
    else if (g.b_col) hipLaunchKernelGGL((k_layer_mm<S, P, false, true, false, T>), grid, block, 0, ctx->stream, g);
    else if (g.gated) hipLaunchKernelGGL((k_layer_mm<S, P, false, false, true, T>), grid, block, 0, ctx->stream, g);
    else hipLaunchKernelGGL((k_layer_mm<S, P, false, false, false, T>), grid, block, 0, ctx->stream, g);
}

template <typename S, int P, typename Large, typename Medium, typename Small, typename Tiny>
gs_status launch_layer_mm(gs_ctx* ctx, const LayerMm& g)
{
    GsTimerScope ts(ctx, "layer_mm");
    if (g.tile == kLarge) launch_mode<S, P, Large>(ctx, g);
    else if (g.tile == kMedium) launch_mode<S, P, Medium>(ctx, g);
    else if (g.tile == kSmall) launch_mode<S, P, Small>(ctx, g);
    else launch_mode<S, P, Tiny>(ctx, g);
    if (g.splits > 1) {
        const dim3 grid((uint32_t)std::min(ceil_div(g.m * ((g.e.n + 3) / 4), 256), kMaxGrid)), block(256);
        if (g.gated) hipLaunchKernelGGL((k_join<S, true>), grid, block, 0, ctx->stream, g);
        else hipLaunchKernelGGL((k_join<S, false>), grid, block, 0, ctx->stream, g);
    }
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

}  // namespace gsm
