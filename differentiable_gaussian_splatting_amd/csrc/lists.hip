// lists.hip -- the global norm of a list of gradients, its clipping, and Adam
// over a list of tensors.
//
//   norm = sqrt(sum over all values of g^2),  c = min(1, max_norm / (norm + 1e-6))
//   clip:  out = c g
//   Adam:  g' = c g, m = b1 m + (1 - b1) g', v = b2 v + (1 - b2) g'^2,
//          p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// A launch takes the descriptors of up to a few dozen tensors as kernel
// arguments (no table is copied to the device).  Each tensor's values are
// split into pieces of `piece` consecutive values, one block per piece; the
// piece is chosen from the list's total so that the blocks fill the device.
// The norm's squares are added in f64: no f32 value overflows or vanishes,
// and one partial per block, summed in a fixed order by every block that needs
// the total, makes the result independent of timing.
#include "gs_device.h"
#include "gs_internal.h"
#include "gs_tensor.h"

#include <algorithm>
#include <type_traits>

namespace {

constexpr int kThreads = 256;

// Where a tensor's rows are apart: value k of its flat order is value k % cols
// of row k / cols.  The tensors of a launch share a short table of these; a
// tensor's `apart` is its place in it, or -1: its rows follow one another.
struct Apart {
    int64_t stride, ostride;
    uint32_t cols;
    uint32_t pad;
};
constexpr int kApart = 16;

// the fields of a launch's tensor that every kernel needs
struct Common {
    int64_t n;
    uint32_t bend;      // blocks of the tensors up to and including this one
    int8_t type, type2, apart, pad;
};

struct NormTensor {
    Common c;
    const void* p;
};
struct ScaleTensor {
    Common c;
    const void* p;
    void* o;
};
struct AdamTensor {
    Common c;
    float *p, *m, *v;
    const void* g;
    void* copy;
};

// kernel arguments, within 4 KB
template <typename T, int CAP>
struct Job {
    static constexpr int kCap = CAP;
    T t[CAP];
    Apart apart[kApart];
    int64_t piece;
    int32_t count, aparts;
};
typedef Job<NormTensor, 144> NormJob;
typedef Job<ScaleTensor, 108> ScaleJob;
typedef Job<AdamTensor, 62> AdamJob;
static_assert(sizeof(NormJob) <= 3968 && sizeof(ScaleJob) <= 3968 && sizeof(AdamJob) <= 3968, "kernel arguments");

struct AdamConst {
    float b1, b2, c1, c2;   // betas and 1 - betas
    float rate;             // lr / (1 - b1^t)
    float inv2;             // 1 / (1 - b2^t)
    float eps, keep;        // keep = 1 - lr weight_decay
};

// the tensor of this block and its piece [k0, k1)
template <typename J>
__device__ __forceinline__ int piece_of_block(const J& job, int64_t& k0, int64_t& k1)
{
    const uint32_t b = blockIdx.x;
    int lo = 0, hi = job.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (b < job.t[mid].c.bend) hi = mid;
        else lo = mid + 1;
    }
    k0 = (int64_t)(b - (lo ? job.t[lo - 1].c.bend : 0u)) * job.piece;
    k1 = min(job.t[lo].c.n, k0 + job.piece);
    return lo;
}

// f(k, place) for every value k of [k0, k1) of a tensor whose rows are apart;
// place: its offset with row stride `stride`, place2 with `ostride`.  The
// first row is divided for once, the rest in 32 bits (a piece is < 2^31).
template <typename F>
__device__ __forceinline__ void each_apart(const Apart& a, int64_t k0, int64_t k1, F&& f)
{
    const int64_t row0 = k0 / a.cols;
    const uint32_t rem = (uint32_t)(k0 - row0 * a.cols);
    for (uint32_t j = threadIdx.x; j < (uint32_t)(k1 - k0); j += kThreads) {
        const uint32_t r = (rem + j) / a.cols, c = (rem + j) - r * a.cols;
        f(k0 + j, (row0 + r) * a.stride + c, (row0 + r) * a.ostride + c);
    }
}

__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double sh[kThreads / 64];
    v = gsd::wave_sum_d(v);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < kThreads / 64; ++w) s += sh[w];
    __syncthreads();
    return s;
}

// sum of the partials, the same in every block
__device__ __forceinline__ double total_of(const double* __restrict__ part, int64_t n)
{
    double s = 0.0;
    for (int64_t k = threadIdx.x; k < n; k += kThreads) s += part[k];
    return block_sum(s);
}

__device__ __forceinline__ float factor_of(double norm, double max_norm)
{
    if (max_norm == __builtin_inf() && norm < __builtin_inf()) return 1.0f;
    const double c = max_norm / (norm + 1e-6);
    return (float)(c > 1.0 ? 1.0 : c);   // NaN stays
}

// Sum of squares of a piece: four packs of 16 bytes per thread in flight.
template <typename T>
__device__ __forceinline__ double squares(const T* __restrict__ p, int64_t n)
{
    constexpr int V = 16 / sizeof(T), U = 4;
    double s = 0.0;
    int64_t k = (int64_t)threadIdx.x * V;
    auto add = [&](const gst::Pack<T, V>& x) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const double d = (double)(float)x.v[e];
            s = __builtin_fma(d, d, s);
        }
    };
    for (; k + (U - 1) * kThreads * V + V <= n; k += U * kThreads * V) {
        gst::Pack<T, V> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = gst::load<T, V>(p + k + u * kThreads * V);
#pragma unroll
        for (int u = 0; u < U; ++u) add(x[u]);
    }
    for (; k + V <= n; k += kThreads * V) add(gst::load<T, V>(p + k));
    const int64_t t = n / V * V + threadIdx.x;
    if (t < n) {
        const double d = (double)(float)p[t];
        s = __builtin_fma(d, d, s);
    }
    return s;
}

__global__ __launch_bounds__(kThreads) void k_squares(NormJob job, double* __restrict__ part)
{
    int64_t k0, k1;
    const NormTensor& t = job.t[piece_of_block(job, k0, k1)];
    double s = 0.0;
    auto typed = [&](auto x) {
        using T = decltype(x);
        const T* p = (const T*)t.p;
        if (t.c.apart < 0) s = squares<T>(p + k0, k1 - k0);
        else
            each_apart(job.apart[t.c.apart], k0, k1, [&](int64_t, int64_t at, int64_t) {
                const double d = (double)(float)p[at];
                s = __builtin_fma(d, d, s);
            });
    };
    if (t.c.type == GS_F32) typed(float{});
    else if (t.c.type == GS_F16) typed(gst::f16{});
    else typed(gst::bf16{});
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void k_norm(const double* __restrict__ part, int64_t n, double max_norm,
                                                   float* __restrict__ norm)
{
    const double s = sqrt(total_of(part, n));
    if (threadIdx.x == 0) {
        norm[0] = (float)s;
        norm[1] = factor_of(s, max_norm);
    }
}

template <typename T>
__device__ __forceinline__ void scale(const T* p, T* o, int64_t n, float c)
{
    constexpr int V = 16 / sizeof(T), U = 4;
    int64_t k = (int64_t)threadIdx.x * V;
    auto put = [&](int64_t at, const gst::Pack<T, V>& x) {
        gst::Pack<T, V> y;
#pragma unroll
        for (int e = 0; e < V; ++e) y.v[e] = gst::narrow<T>(c * (float)x.v[e]);
        gst::store<T, V>(o + at, y);
    };
    for (; k + (U - 1) * kThreads * V + V <= n; k += U * kThreads * V) {
        gst::Pack<T, V> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = gst::load<T, V>(p + k + u * kThreads * V);
#pragma unroll
        for (int u = 0; u < U; ++u) put(k + u * kThreads * V, x[u]);
    }
    for (; k + V <= n; k += kThreads * V) put(k, gst::load<T, V>(p + k));
    const int64_t t = n / V * V + threadIdx.x;
    if (t < n) o[t] = gst::narrow<T>(c * (float)p[t]);
}

// Every block adds the norm's partials itself, in one order (a launch less
// than a norm of its own); the first one writes the norm.
__global__ __launch_bounds__(kThreads) void k_scale(ScaleJob job, const double* __restrict__ part, int64_t parts,
                                                    double max_norm, float* __restrict__ norm)
{
    const double total = sqrt(total_of(part, parts));
    const float c = factor_of(total, max_norm);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) {
        norm[0] = (float)total;
        norm[1] = c;
    }
    int64_t k0, k1;
    const ScaleTensor& t = job.t[piece_of_block(job, k0, k1)];
    if (c == 1.0f && t.o == t.p) return;
    auto typed = [&](auto x) {
        using T = decltype(x);
        const T* p = (const T*)t.p;
        T* o = (T*)t.o;
        if (t.c.apart < 0) scale<T>(p + k0, o + k0, k1 - k0, c);
        else
            each_apart(job.apart[t.c.apart], k0, k1, [&](int64_t, int64_t at, int64_t to) {
                o[to] = gst::narrow<T>(c * (float)p[at]);
            });
    };
    if (t.c.type == GS_F32) typed(float{});
    else if (t.c.type == GS_F16) typed(gst::f16{});
    else typed(gst::bf16{});
}

__device__ __forceinline__ void adam_value(float g, float& p, float& m, float& v, const AdamConst& a)
{
    m = a.b1 * m + a.c1 * g;
    v = a.b2 * v + a.c2 * (g * g);
    p = a.keep * p - a.rate * m / (sqrtf(v * a.inv2) + a.eps);
}

__device__ __forceinline__ void put_copy(const AdamTensor& t, int64_t k, float p)
{
    if (t.c.type2 == GS_F32) ((float*)t.copy)[k] = p;
    else if (t.c.type2 == GS_F16) ((gst::f16*)t.copy)[k] = gst::narrow<gst::f16>(p);
    else ((gst::bf16*)t.copy)[k] = gst::narrow<gst::bf16>(p);
}

// A piece: packs of four values, two in flight per thread (p, m, v of 16 bytes
// each and the gradient's).
template <typename T>
__device__ __forceinline__ void adam(const AdamTensor& t, int64_t k0, int64_t n, float c, const AdamConst& a)
{
    constexpr int V = 4, U = 2;
    float *pp = t.p + k0, *mp = t.m + k0, *vp = t.v + k0;
    const T* gp = (const T*)t.g + k0;
    auto go = [&](int64_t k, auto count) {
        constexpr int N = decltype(count)::value;
        gst::Pack<float, V> p[N], m[N], v[N];
        gst::Pack<T, V> g[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int64_t at = k + u * kThreads * V;
            p[u] = gst::load<float, V>(pp + at);
            m[u] = gst::load<float, V>(mp + at);
            v[u] = gst::load<float, V>(vp + at);
            g[u] = gst::load<T, V>(gp + at);
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int64_t at = k + u * kThreads * V;
#pragma unroll
            for (int e = 0; e < V; ++e) adam_value(c * (float)g[u].v[e], p[u].v[e], m[u].v[e], v[u].v[e], a);
            gst::store<float, V>(pp + at, p[u]);
            gst::store<float, V>(mp + at, m[u]);
            gst::store<float, V>(vp + at, v[u]);
            if (t.copy) {
                auto low = [&](auto x) {
                    using O = decltype(x);
                    gst::Pack<O, V> y;
#pragma unroll
                    for (int e = 0; e < V; ++e) y.v[e] = gst::narrow<O>(p[u].v[e]);
                    gst::store<O, V>((O*)t.copy + k0 + at, y);
                };
                if (t.c.type2 == GS_F32) low(float{});
                else if (t.c.type2 == GS_F16) low(gst::f16{});
                else low(gst::bf16{});
            }
        }
    };
    int64_t k = (int64_t)threadIdx.x * V;
    for (; k + (U - 1) * kThreads * V + V <= n; k += U * kThreads * V) go(k, std::integral_constant<int, U>{});
    for (; k + V <= n; k += kThreads * V) go(k, std::integral_constant<int, 1>{});
    const int64_t r = n / V * V + threadIdx.x;
    if (r < n) {
        float p = pp[r], m = mp[r], v = vp[r];
        adam_value(c * (float)gp[r], p, m, v, a);
        pp[r] = p;
        mp[r] = m;
        vp[r] = v;
        if (t.copy) put_copy(t, k0 + r, p);
    }
}

__global__ __launch_bounds__(kThreads) void k_adam_list(AdamJob job, AdamConst a, const float* __restrict__ norm)
{
    float c = 1.0f;
    if (norm) {
        if (!(fabsf(norm[0]) < __builtin_inff())) return;   // not finite
        c = norm[1];
    }
    int64_t k0, k1;
    const AdamTensor& t = job.t[piece_of_block(job, k0, k1)];
    auto typed = [&](auto x) {
        using T = decltype(x);
        if (t.c.apart < 0) adam<T>(t, k0, k1 - k0, c, a);
        else
            each_apart(job.apart[t.c.apart], k0, k1, [&](int64_t k, int64_t at, int64_t) {
                float p = t.p[k], m = t.m[k], v = t.v[k];
                adam_value(c * (float)((const T*)t.g)[at], p, m, v, a);
                t.p[k] = p;
                t.m[k] = m;
                t.v[k] = v;
                if (t.copy) put_copy(t, k, p);
            });
    };
    if (t.c.type == GS_F32) typed(float{});
    else if (t.c.type == GS_F16) typed(gst::f16{});
    else typed(gst::bf16{});
}

// rows x cols values that lie one after the other
bool dense(const gs_tensor& t) { return t.rows <= 1 || t.stride == t.cols; }

// values per block for `total` values: about eight blocks of 256 threads per
// compute unit, at least 1024 values
int64_t piece_of(const gs_ctx* ctx, int64_t total)
{
    const int64_t p = ceil_div(total, (int64_t)ctx->num_cu * 8);
    return std::max<int64_t>(1024, ceil_div(p, 1024) * 1024);
}

int64_t values(const gs_tensor* t, int32_t n)
{
    int64_t s = 0;
    for (int32_t k = 0; k < n; ++k) s += t[k].rows * t[k].cols;
    return s;
}

int64_t pieces(const gs_tensor* t, int32_t n, int64_t piece)
{
    int64_t s = 0;
    for (int32_t k = 0; k < n; ++k) s += ceil_div(t[k].rows * t[k].cols, piece);
    return s;
}

// Splits the tensors with values over launches of at most a job's
// descriptors (and kApart of rows apart): put(descriptor, tensor index) fills
// in the pointers, go(job, blocks) launches.  in, out: the tensors whose rows
// may be apart (out may be null).
template <typename J, typename P, typename G>
void each_launch(const gs_tensor* in, const gs_tensor* out, int32_t n, int64_t piece, P&& put, G&& go)
{
    J job;
    job.piece = piece;
    job.count = job.aparts = 0;
    uint32_t blocks = 0;
    auto flush = [&]() {
        if (job.count) go(job, blocks);
        job.count = job.aparts = 0;
        blocks = 0;
    };
    for (int32_t k = 0; k < n; ++k) {
        const gs_tensor& t = in[k];
        const int64_t values = t.rows * t.cols;
        if (values == 0) continue;
        const bool apart = !dense(t) || (out && !dense(out[k]));
        if (job.count == J::kCap || (apart && job.aparts == kApart)) flush();
        blocks += (uint32_t)ceil_div(values, piece);
        auto& d = job.t[job.count++];
        d.c.n = values;
        d.c.bend = blocks;
        d.c.type = (int8_t)t.type;
        d.c.type2 = 0;
        d.c.apart = -1;
        if (apart) {
            d.c.apart = (int8_t)job.aparts;
            job.apart[job.aparts++] = Apart{t.stride, out ? out[k].stride : 0, (uint32_t)t.cols, 0};
        }
        put(d, k);
    }
    flush();
}

// the partials of a list's squares, one per block
gs_status squares_of(gs_ctx* ctx, const gs_tensor* grads, int32_t n, std::vector<GsAlloc>* tmp, double** part,
                     int64_t* parts)
{
    const int64_t piece = piece_of(ctx, values(grads, n));
    *parts = pieces(grads, n, piece);
    *part = (double*)gs_malloc(ctx, 8 * std::max<int64_t>(*parts, 1), GS_MEM_SCRATCH, tmp);
    if (!*part) return GS_ERR_OOM;
    GsTimerScope ts(ctx, "grad_norm");
    int64_t base = 0;
    each_launch<NormJob>(grads, nullptr, n, piece, [&](NormTensor& d, int32_t k) { d.p = grads[k].data; },
                         [&](const NormJob& job, uint32_t nb) {
                             hipLaunchKernelGGL(k_squares, dim3(nb), dim3(kThreads), 0, ctx->stream, job, *part + base);
                             base += nb;
                         });
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

}  // namespace

gs_status launch_grad_norm(gs_ctx* ctx, const gs_tensor* grads, int32_t n, double max_norm, float* norm,
                           std::vector<GsAlloc>* tmp)
{
    double* part;
    int64_t parts;
    const gs_status st = squares_of(ctx, grads, n, tmp, &part, &parts);
    if (st != GS_OK) return st;
    GsTimerScope ts(ctx, "grad_norm");
    hipLaunchKernelGGL(k_norm, dim3(1), dim3(kThreads), 0, ctx->stream, part, parts, max_norm, norm);
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

gs_status launch_clip(gs_ctx* ctx, const gs_tensor* in, int32_t n, double max_norm, const gs_tensor* out, float* norm,
                      std::vector<GsAlloc>* tmp)
{
    const int64_t total = values(in, n);
    if (total == 0) return launch_grad_norm(ctx, in, n, max_norm, norm, tmp);
    double* part;
    int64_t parts;
    const gs_status st = squares_of(ctx, in, n, tmp, &part, &parts);
    if (st != GS_OK) return st;
    GsTimerScope ts(ctx, "clip");
    float* write = norm;   // by the first launch
    each_launch<ScaleJob>(in, out, n, piece_of(ctx, total),
                          [&](ScaleTensor& d, int32_t k) {
                              d.p = in[k].data;
                              d.o = out[k].data;
                          },
                          [&](const ScaleJob& job, uint32_t nb) {
                              hipLaunchKernelGGL(k_scale, dim3(nb), dim3(kThreads), 0, ctx->stream, job, part, parts,
                                                 max_norm, write);
                              write = nullptr;
                          });
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

gs_status launch_adam_list(gs_ctx* ctx, const gs_tensor* p, const gs_tensor* m, const gs_tensor* v, const gs_tensor* g,
                           const gs_tensor* copies, int32_t n, const gs_adam_opts* o, const float* norm)
{
    AdamConst a;
    a.b1 = (float)o->beta1;
    a.b2 = (float)o->beta2;
    a.c1 = (float)(1.0 - o->beta1);
    a.c2 = (float)(1.0 - o->beta2);
    a.rate = (float)(o->lr / (1.0 - std::pow(o->beta1, (double)o->step)));
    a.inv2 = (float)(1.0 / (1.0 - std::pow(o->beta2, (double)o->step)));
    a.eps = (float)o->eps;
    a.keep = (float)(1.0 - o->lr * o->weight_decay);
    GsTimerScope ts(ctx, "adam_list");
    each_launch<AdamJob>(g, nullptr, n, piece_of(ctx, values(g, n)),
                         [&](AdamTensor& d, int32_t k) {
                             d.p = (float*)p[k].data;
                             d.m = (float*)m[k].data;
                             d.v = (float*)v[k].data;
                             d.g = g[k].data;
                             d.copy = copies ? copies[k].data : nullptr;
                             d.c.type2 = (int8_t)(copies ? copies[k].type : 0);
                         },
                         [&](const AdamJob& job, uint32_t nb) {
                             hipLaunchKernelGGL(k_adam_list, dim3(nb), dim3(kThreads), 0, ctx->stream, job, a, norm);
                         });
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}
