// layers.h -- what the files of the layer operators share: activations, the
// description of one matrix product with its epilogue, and its launch.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gs_internal.h"
#include "layer_plan.h"
#include "mm.h"

namespace gsm {

// z sigma(v) and its slope, sigma(v) + z sigma(v) sigma(-v) v', with v = z
// (silu), v = 2 sqrt(2 / pi) (z + 0.044715 z^3) (gelu).  With q = exp(-|v|) and
// r = 1 / (1 + q), sigma is r or q r and sigma(v) sigma(-v) = q r^2: no
// difference of near numbers.  Where q vanishes the value is z or 0, the slope
// 1 or 0, at infinities too.
constexpr float kGelu1 = 1.5957691216057308f, kGelu3 = 0.044715f;

struct Sigma {
    float p, t;   // sigma(v), sigma(v) sigma(-v)
};
// The hardware's exponential and reciprocal are within an ulp or so; rounding
// the exponent's argument costs |v| 2^-24 of q, where q itself is exp(-|v|).
// (With expf and a division an activation costs 40 operations, not 10: 1M rows
// of 64 silu values 52 us.)
__device__ __forceinline__ Sigma sigma(float v)
{
    const float q = __builtin_amdgcn_exp2f(-fabsf(v) * 1.44269504f), r = __builtin_amdgcn_rcpf(1.0f + q);
    return Sigma{v >= 0.0f ? r : q * r, q * r * r};
}
__device__ __forceinline__ float gelu_arg(float z) { return kGelu1 * (z + kGelu3 * z * z * z); }

__device__ __forceinline__ float act_value(float z, int act)
{
    if (act == GS_ACT_NONE) return z;
    if (act == GS_ACT_RELU) return z < 0.0f ? 0.0f : z;   // NaN stays
    const Sigma s = sigma(act == GS_ACT_GELU ? gelu_arg(z) : z);
    if (act == GS_ACT_SIGMOID) return s.p;
    return s.p == 0.0f ? 0.0f : z * s.p;
}

// value and slope
__device__ __forceinline__ float2 act_both(float z, int act)
{
    if (act == GS_ACT_NONE) return make_float2(z, 1.0f);
    if (act == GS_ACT_RELU) return make_float2(z < 0.0f ? 0.0f : z, z > 0.0f ? 1.0f : 0.0f);
    const Sigma s = sigma(act == GS_ACT_GELU ? gelu_arg(z) : z);
    if (act == GS_ACT_SIGMOID) return make_float2(s.p, s.t);
    const float dv = act == GS_ACT_GELU ? kGelu1 * (1.0f + 3.0f * kGelu3 * z * z) : 1.0f;
    return make_float2(s.p == 0.0f ? 0.0f : z * s.p, s.t == 0.0f ? s.p : s.p + z * s.t * dv);
}

// f16 operands that may lie beyond f16's range are scaled by 2^e, which brings
// their largest finite |value| to [2^14, 2^15) as far as 2^-e stays a normal float.
__device__ __forceinline__ int scale_exponent(float most)
{
    return most > 0.0f ? min(15 - __builtin_amdgcn_frexp_expf(most), 126) : 0;
}
__device__ __forceinline__ float larger(float most, float v)
{
    const float a = fabsf(v);
    return a <= 3.402823466e38f ? fmaxf(most, a) : most;   // not infinity, not NaN
}

// What follows a product: out = act(z + bias) + residual, with z + bias kept
// in pre (each null: not there).  Types are GS_F32 or the product's own.  down:
// what the row's sums are multiplied with first, at m lddown.
struct Epilogue {
    const void* bias;
    const void* res;
    void* pre;
    void* out;
    int64_t ldres, ldpre, ldout;
    int64_t n;                   // columns of out
    int32_t act;
    int8_t bias_type, res_type, pre_type, out_type;
    const float* down;
    int64_t lddown;
};

struct LayerMm {
    Operand a, b;                // rows of out, columns of out
    int64_t m, k;
    Epilogue e;
    int64_t tm, tn;              // tiles
    int64_t full;                // the first `full` tiles are formed whole, each by one block;
    int32_t splits, tile;        // the others in `splits` ranges of kper values of k,
    int64_t kper;                // a multiple of the tile's step,
    float* ws;                   // whose sums are kept here: [splits][tiles - full][rows][columns of a tile]
    bool a_col, b_col, gated;    // a_col only with b_col
    const void* a_other;         // what a is instead of a.p if *other is not 0 (other null: it stays)
    const int32_t* other;
};

// Whether the tiles of a product of 16-bit operands load straight into LDS
// (Direct in mm.h): rows that start on 16 bytes, and for an operand whose k runs
// down the columns a multiple of 8 columns, so that a tile moved back to end
// with them still starts on 16 bytes.
inline bool loads_direct(const LayerMm& g)
{
    const auto fits = [](const Operand& o, bool col) {
        return (uintptr_t)o.p % 16 == 0 && o.ld % 8 == 0 && !(col && o.rows % 8);
    };
    return fits(g.a, g.a_col) && fits(g.b, g.b_col);
}

// one type each (layer_mm_*.hip)
gs_status launch_layer_mm_f32(gs_ctx* ctx, const LayerMm& g);
gs_status launch_layer_mm_f16(gs_ctx* ctx, const LayerMm& g);
gs_status launch_layer_mm_bf16(gs_ctx* ctx, const LayerMm& g);
// dx and dw of kSmall tiles in one launch
gs_status launch_layer_pair_f32(gs_ctx* ctx, const LayerMm& x, const LayerMm& w);
gs_status launch_layer_pair_f16(gs_ctx* ctx, const LayerMm& x, const LayerMm& w);
gs_status launch_layer_pair_bf16(gs_ctx* ctx, const LayerMm& x, const LayerMm& w);
// x w^T of few rows (layer_few.hip)
bool few_rows(const LayerMm& g);
gs_status launch_layer_few(gs_ctx* ctx, int type, const LayerMm& g);

typedef Tile<256, 256, 64, 2, 4, 2> Large16;
typedef Tile<128, 128, 64, 2, 2, 2> Medium16;
typedef Tile<64, 64, 64, 2, 2, 2> Small16;
typedef Tile<64, 64, 64, 2, 2, 2, true> Tiny16;
typedef Tile<256, 128, 32, 4, 2, 2> Large32;
typedef Tile<128, 128, 32, 2, 2, 1> Medium32;
typedef Tile<64, 64, 32, 2, 2, 2> Small32;
typedef Tile<64, 64, 32, 2, 2, 2, true> Tiny32;

template <typename T>
constexpr bool planned_as(const TileCost& c)
{
    return c.m == T::BM && c.n == T::BN && c.k == T::BK;
}
static_assert(planned_as<Large16>(kCost16[kLarge]) && planned_as<Large16>(kCostDirect[kLarge]) &&
              planned_as<Medium16>(kCost16[kMedium]) && planned_as<Medium16>(kCostDirect[kMedium]) &&
              planned_as<Small16>(kCost16[kSmall]) && planned_as<Small16>(kCostDirect[kSmall]) &&
              planned_as<Tiny16>(kCost16[kTiny]) && planned_as<Tiny16>(kCostDirect[kTiny]) &&
              planned_as<Large32>(kCost32[kLarge]) && planned_as<Medium32>(kCost32[kMedium]) &&
              planned_as<Small32>(kCost32[kSmall]) && planned_as<Tiny32>(kCost32[kTiny]), "tiles and their costs");

}  // namespace gsm
