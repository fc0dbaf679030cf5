// gs_tensor.h -- device-side helpers of the tensor-list and table kernels:
// element types and loads and stores of several values at once.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gst {

typedef _Float16 f16;
typedef __bf16 bf16;

// N values in memory, aligned to the element only: rows of odd widths, columns
// of wider rows and views into flat buffers start anywhere.  The compiler
// loads and stores a pack of up to 16 bytes in one instruction whatever its
// alignment (gfx950 global memory takes any).
template <typename T, int N>
struct Pack {
    T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load(const T* p)
{
    Pack<T, N> r;
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
}

template <typename T, int N>
__device__ __forceinline__ void store(T* p, const Pack<T, N>& r)
{
    __builtin_memcpy(p, &r, sizeof(r));
}

// store of values that are not read again soon
template <typename T, int N>
__device__ __forceinline__ void store_once(T* p, const Pack<T, N>& r)
{
    typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
    typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(2)));
    if constexpr (sizeof(r) == 16) __builtin_nontemporal_store(__builtin_bit_cast(v4, r), reinterpret_cast<v4*>(p));
    else if constexpr (sizeof(r) == 8) __builtin_nontemporal_store(__builtin_bit_cast(v2, r), reinterpret_cast<v2*>(p));
    else store(p, r);
}

// x rounded to T (to nearest, ties to even).  For f16 the compiler would fuse a
// product before the conversion into a multiply-add with +0, which turns -0
// into +0; the empty statement keeps the two apart.
template <typename T>
__device__ __forceinline__ T narrow(float x)
{
    if constexpr (sizeof(T) == 2) asm("" : "+v"(x));
    return (T)x;
}

// idx[i] as a row of a table, or `rows` (a value no row has) when it is outside
// [0, rows) or equal to skip
template <typename I>
__device__ __forceinline__ uint32_t row_of(const I* __restrict__ idx, int64_t i, uint32_t rows, int64_t skip)
{
    const int64_t v = (int64_t)idx[i];
    return v >= 0 && v < (int64_t)rows && v != skip ? (uint32_t)v : rows;
}

// Calls f with a value of the element type (GS_F32, GS_F16, GS_BF16).
template <typename F>
inline void with_type(int type, F&& f)
{
    if (type == 0) f(float{});
    else if (type == 1) f(f16{});
    else f(bf16{});
}

}  // namespace gst
