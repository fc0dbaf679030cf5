// lists.hip -- the global norm of a list of gradients, its clipping, and Adam
// over a list of tensors.
//
//   norm = sqrt(sum over all values of g^2),  c = min(1, max_norm / (norm + 1e-6))
//   clip:  out = c g
//   Adam:  g' = c g, m = b1 m + (1 - b1) g', v = b2 v + (1 - b2) g'^2,
//          p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// A launch takes the descriptors of up to a few dozen tensors as kernel
// arguments (no copy of a table to the device).  Each tensor's values are
// split into pieces of `piece` consecutive values, one block per piece; the
// piece is chosen from the list's total so that the blocks fill the device.
// The norm's squares are added in f64: no f32 value overflows or vanishes,
// and one partial per block, summed in a fixed order by every block that needs
// the total, makes the result independent of timing.
#include "gs_device.h"
#include "gs_internal.h"
#include "gs_tensor.h"

namespace {

constexpr int kThreads = 256;

// value k of a tensor in flat order; cols = 0: its rows follow one another
__device__ __forceinline__ int64_t at(int64_t k, uint32_t cols, int64_t stride)
{
    if (cols == 0) return k;
    const int64_t r = k / cols;
    return r * stride + (k - r * cols);
}

struct NormTensor {
    const void* p;
    int64_t n, stride;
    uint32_t cols;
    int32_t type;
};
constexpr int kNormTensors = 96;
struct NormJob {
    NormTensor t[kNormTensors];
    uint32_t bend[kNormTensors];   // blocks of the tensors up to and including each
    int32_t count;
    int64_t piece;
};

struct ScaleTensor {
    const void* p;
    void* o;
    int64_t n, stride, ostride;
    uint32_t cols;
    int32_t type;
};
constexpr int kScaleTensors = 64;
struct ScaleJob {
    ScaleTensor t[kScaleTensors];
    uint32_t bend[kScaleTensors];
    int32_t count;
    int64_t piece;
};

struct AdamTensor {
    float *p, *m, *v;
    const void* g;
    void* copy;
    int64_t n, stride;
    uint32_t cols;
    int16_t type, ctype;
};
constexpr int kAdamTensors = 52;
struct AdamListJob {
    AdamTensor t[kAdamTensors];
    uint32_t bend[kAdamTensors];
    int32_t count;
    int64_t piece;
};

struct AdamConst {
    float b1, b2, c1, c2;   // betas and 1 - betas
    float rate;             // lr / (1 - b1^t)
    float inv2;             // 1 / (1 - b2^t)
    float eps, keep;        // keep = 1 - lr weight_decay
};

// the tensor of block b: the first whose bend exceeds it
template <typename J>
__device__ __forceinline__ int tensor_of(const J& job, uint32_t b)
{
    int lo = 0, hi = job.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (b < job.bend[mid]) hi = mid;
        else lo = mid + 1;
    }
    return lo;
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

template <typename T>
__device__ __forceinline__ double squares(const NormTensor& t, int64_t k0, int64_t k1)
{
    const T* p = (const T*)t.p;
    double s = 0.0;
    for (int64_t k = k0 + threadIdx.x; k < k1; k += kThreads) {
        const double x = (double)(float)p[at(k, t.cols, t.stride)];
        s += x * x;
    }
    return s;
}

__global__ __launch_bounds__(kThreads) void k_squares(NormJob job, double* __restrict__ part)
{
    const int q = tensor_of(job, blockIdx.x);
    const NormTensor& t = job.t[q];
    const int64_t k0 = (int64_t)(blockIdx.x - (q ? job.bend[q - 1] : 0)) * job.piece;
    const int64_t k1 = min(t.n, k0 + job.piece);
    double s;
    if (t.type == GS_F32) s = squares<float>(t, k0, k1);
    else if (t.type == GS_F16) s = squares<gst::f16>(t, k0, k1);
    else s = squares<gst::bf16>(t, k0, k1);
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
__device__ __forceinline__ void scale(const ScaleTensor& t, int64_t k0, int64_t k1, float c)
{
    const T* p = (const T*)t.p;
    T* o = (T*)t.o;
    for (int64_t k = k0 + threadIdx.x; k < k1; k += kThreads)
        o[at(k, t.cols, t.ostride)] = gst::narrow<T>(c * (float)p[at(k, t.cols, t.stride)]);
}

__global__ __launch_bounds__(kThreads) void k_scale(ScaleJob job, const float* __restrict__ norm)
{
    const float c = norm[1];
    const int q = tensor_of(job, blockIdx.x);
    const ScaleTensor& t = job.t[q];
    if (c == 1.0f && t.o == t.p) return;
    const int64_t k0 = (int64_t)(blockIdx.x - (q ? job.bend[q - 1] : 0)) * job.piece;
    const int64_t k1 = min(t.n, k0 + job.piece);
    if (t.type == GS_F32) scale<float>(t, k0, k1, c);
    else if (t.type == GS_F16) scale<gst::f16>(t, k0, k1, c);
    else scale<gst::bf16>(t, k0, k1, c);
}

__device__ __forceinline__ void adam_value(float g, float& p, float& m, float& v, const AdamConst& a)
{
    m = a.b1 * m + a.c1 * g;
    v = a.b2 * v + a.c2 * (g * g);
    p = a.keep * p - a.rate * m / (sqrtf(v * a.inv2) + a.eps);
}

template <typename T>
__device__ __forceinline__ void adam(const AdamTensor& t, int64_t k0, int64_t k1, float c, const AdamConst& a)
{
    for (int64_t k = k0 + threadIdx.x; k < k1; k += kThreads) {
        float p = t.p[k], m = t.m[k], v = t.v[k];
        adam_value(c * (float)((const T*)t.g)[at(k, t.cols, t.stride)], p, m, v, a);
        t.p[k] = p;
        t.m[k] = m;
        t.v[k] = v;
        if (t.copy) {
            if (t.ctype == GS_F32) ((float*)t.copy)[k] = p;
            else if (t.ctype == GS_F16) ((gst::f16*)t.copy)[k] = (gst::f16)p;
            else ((gst::bf16*)t.copy)[k] = (gst::bf16)p;
        }
    }
}

__global__ __launch_bounds__(kThreads) void k_adam_list(AdamListJob job, AdamConst a, const float* __restrict__ norm)
{
    float c = 1.0f;
    if (norm) {
        if (!(fabsf(norm[0]) < __builtin_inff())) return;   // not finite
        c = norm[1];
    }
    const int q = tensor_of(job, blockIdx.x);
    const AdamTensor& t = job.t[q];
    const int64_t k0 = (int64_t)(blockIdx.x - (q ? job.bend[q - 1] : 0)) * job.piece;
    const int64_t k1 = min(t.n, k0 + job.piece);
    if (t.type == GS_F32) adam<float>(t, k0, k1, c, a);
    else if (t.type == GS_F16) adam<gst::f16>(t, k0, k1, c, a);
    else adam<gst::bf16>(t, k0, k1, c, a);
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

// Splits the tensors with values over launches of at most `cap` descriptors:
// put(job.t[k], tensor index) fills a descriptor, go(job, blocks) launches.
template <typename J, typename P, typename G>
void each_launch(const gs_tensor* t, int32_t n, int cap, int64_t piece, P&& put, G&& go)
{
    J job;
    job.piece = piece;
    job.count = 0;
    uint32_t blocks = 0;
    for (int32_t k = 0; k < n; ++k) {
        const int64_t nb = ceil_div(t[k].rows * t[k].cols, piece);
        if (nb == 0) continue;
        put(job.t[job.count], k);
        blocks += (uint32_t)nb;
        job.bend[job.count] = blocks;
        if (++job.count == cap) {
            go(job, blocks);
            job.count = 0;
            blocks = 0;
        }
    }
    if (job.count) go(job, blocks);
}

}  // namespace

gs_status launch_grad_norm(gs_ctx* ctx, const gs_tensor* grads, int32_t n, double max_norm, float* norm,
                           std::vector<GsAlloc>* tmp)
{
    const int64_t piece = piece_of(ctx, values(grads, n)), blocks = pieces(grads, n, piece);
    double* part = (double*)gs_malloc(ctx, 8 * std::max<int64_t>(blocks, 1), GS_MEM_SCRATCH, tmp);
    if (!part) return GS_ERR_OOM;
    {
        GsTimerScope ts(ctx, "grad_norm");
        int64_t base = 0;
        each_launch<NormJob>(grads, n, kNormTensors, piece,
            [&](NormTensor& d, int32_t k) {
                const gs_tensor& g = grads[k];
                d = NormTensor{g.data, g.rows * g.cols, g.stride, dense(g) ? 0u : (uint32_t)g.cols, g.type};
            },
            [&](const NormJob& job, uint32_t nb) {
                hipLaunchKernelGGL(k_squares, dim3(nb), dim3(kThreads), 0, ctx->stream, job, part + base);
                base += nb;
            });
    }
    GsTimerScope ts(ctx, "grad_norm");
    hipLaunchKernelGGL(k_norm, dim3(1), dim3(kThreads), 0, ctx->stream, part, blocks, max_norm, norm);
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

gs_status launch_scale_list(gs_ctx* ctx, const gs_tensor* in, const gs_tensor* out, int32_t n, const float* norm)
{
    GsTimerScope ts(ctx, "clip");
    each_launch<ScaleJob>(in, n, kScaleTensors, piece_of(ctx, values(in, n)),
        [&](ScaleTensor& d, int32_t k) {
            const gs_tensor &g = in[k], &o = out[k];
            d = ScaleTensor{g.data, o.data, g.rows * g.cols, g.stride, o.stride,
                            dense(g) && dense(o) ? 0u : (uint32_t)g.cols, g.type};
        },
        [&](const ScaleJob& job, uint32_t nb) {
            hipLaunchKernelGGL(k_scale, dim3(nb), dim3(kThreads), 0, ctx->stream, job, norm);
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
    each_launch<AdamListJob>(p, n, kAdamTensors, piece_of(ctx, values(p, n)),
        [&](AdamTensor& d, int32_t k) {
            d = AdamTensor{(float*)p[k].data, (float*)m[k].data, (float*)v[k].data, g[k].data,
                           copies ? copies[k].data : nullptr, p[k].rows * p[k].cols, g[k].stride,
                           dense(g[k]) ? 0u : (uint32_t)g[k].cols, (int16_t)g[k].type,
                           (int16_t)(copies ? copies[k].type : 0)};
        },
        [&](const AdamListJob& job, uint32_t nb) {
            hipLaunchKernelGGL(k_adam_list, dim3(nb), dim3(kThreads), 0, ctx->stream, job, a, norm);
        });
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}
