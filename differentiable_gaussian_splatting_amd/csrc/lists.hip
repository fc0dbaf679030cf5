// lists.hip -- the global norm of a list of gradients, its clipping, and Adam
// over a list of tensors.
//
//   norm = sqrt(sum over all values of g^2),  c = min(1, max_norm / (norm + 1e-6))
//   clip:  out = c g
//   Adam:  g' = c g, m = b1 m + (1 - b1) g', v = b2 v + (1 - b2) g'^2,
//          p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// All three are bound by memory.  354M f32 (five tensors of a 6M-Gaussian
// scene): squares 231-271 us (5.2-6.1 TB/s), scaling 451 us (6.3 TB/s), Adam
// 1791 us (9.9 GB, 5.5 TB/s); a plain device copy reaches 4.7 TB/s and an
// update in place 5.9.  Small lists are bound by their launches: 28,000 values
// clipped in 8.2 us (one launch), an Adam step of 23,000 with its norm in 12.4
// (two).
//
// A launch takes the descriptors of dozens of tensors as kernel arguments (no
// table is copied from the host).  Each tensor's values are split into pieces,
// one block per piece.  The norm's squares are added in f64: no f32 value
// overflows or vanishes (the sums stay hidden behind the loads), and one
// partial per block, summed in a fixed order by every block that needs the
// total, makes the result independent of timing.
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
constexpr int kApart = 16;   // in a launch's kernel arguments

// the fields of a launch's tensor that every kernel needs
struct Common {
    int64_t n;
    uint32_t bend;      // blocks of the tensors up to and including this one
    int8_t type, type2;
    int16_t apart;
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

// The descriptors of a launch: in its kernel arguments (within 4 KB), or, for
// large lists that would take more than three such launches, in a table on
// the device that small launches fill from theirs (Adam over 220 tensors of
// 11.3M values: 85 us against 99; over 250 tensors of 0.4M values the table
// costs 4 us).
template <typename T, int CAP>
struct Job {
    typedef T Tensor;
    static constexpr int kCap = CAP;
    T t[CAP];
    Apart apart[kApart];
    int64_t piece;
    int32_t count, aparts;
};
typedef Job<NormTensor, 144> NormJob;
typedef Job<ScaleTensor, 108> ScaleJob;
typedef Job<AdamTensor, 62> AdamJob;
template <typename T>
struct Table {
    const T* t;
    const Apart* apart;
    int64_t piece;
    int32_t count;
};
static_assert(sizeof(NormJob) <= 3968 && sizeof(ScaleJob) <= 3968 && sizeof(AdamJob) <= 3968, "kernel arguments");

struct AdamConst {
    float b1, b2, c1, c2;   // betas and 1 - betas
    float rate;             // lr / (1 - b1^t)
    float inv2;             // 1 / (1 - b2^t)
    float eps, keep;        // keep = 1 - lr weight_decay
};

// the tensor of block b, and that block among the tensor's `blocks`
template <typename J>
__device__ __forceinline__ int tensor_of_block(const J& job, uint32_t b, uint32_t& among, uint32_t& blocks)
{
    int lo = 0, hi = job.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (b < job.t[mid].c.bend) hi = mid;
        else lo = mid + 1;
    }
    const uint32_t before = lo ? job.t[lo - 1].c.bend : 0u;
    among = b - before;
    blocks = job.t[lo].c.bend - before;
    return lo;
}

// For the values k of [k0, k1) of a tensor whose rows are apart:
// use(k, place2, get(k, place)), place its offset with row stride `stride`,
// place2 with `ostride`; a thread gets four values before it uses them.  The
// first row is divided for once, the rest in 32 bits (a piece is < 2^31).
template <typename G, typename F>
__device__ __forceinline__ void each_apart(const Apart& a, int64_t k0, int64_t k1, G&& get, F&& use)
{
    constexpr int U = 4;
    const int64_t row0 = k0 / a.cols;
    const uint32_t rem = (uint32_t)(k0 - row0 * a.cols), n = (uint32_t)(k1 - k0);
    auto run = [&](uint32_t j, auto count) {
        constexpr int N = decltype(count)::value;
        int64_t row[N];
        uint32_t c[N];
        decltype(get(int64_t{}, int64_t{})) x[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint32_t i = rem + j + u * kThreads, r = i / a.cols;
            row[u] = row0 + r;
            c[u] = i - r * a.cols;
            x[u] = get(k0 + j + u * kThreads, row[u] * a.stride + c[u]);
        }
#pragma unroll
        for (int u = 0; u < N; ++u) use(k0 + j + u * kThreads, row[u] * a.ostride + c[u], x[u]);
    };
    uint32_t j = threadIdx.x;
    for (; j + (U - 1) * kThreads < n; j += U * kThreads) run(j, std::integral_constant<int, U>{});
    for (; j < n; j += kThreads) run(j, std::integral_constant<int, 1>{});
}

// a job's descriptors into a table
template <typename J>
__global__ __launch_bounds__(kThreads) void k_fill_table(J job, typename J::Tensor* __restrict__ t,
                                                         Apart* __restrict__ apart)
{
    for (int k = threadIdx.x; k < job.count; k += kThreads) t[k] = job.t[k];
    for (int k = threadIdx.x; k < job.aparts; k += kThreads) apart[k] = job.apart[k];
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

// Sum of squares of the block's share of a tensor: every `blocks`-th run of
// four packs per thread, so that all blocks together walk through memory from
// front to back (354M f32 within a clip: 231 us, 270 with a contiguous piece
// per block).
template <typename T>
__device__ __forceinline__ double squares(const T* __restrict__ p, int64_t n, uint32_t among, uint32_t blocks)
{
    constexpr int V = 16 / sizeof(T), U = 4, kRun = kThreads * V * U;
    double s = 0.0;
    auto add = [&](const gst::Pack<T, V>& x) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const double d = (double)(float)x.v[e];
            s = __builtin_fma(d, d, s);
        }
    };
    int64_t k = (int64_t)among * kRun;
    for (; k + kRun <= n; k += (int64_t)blocks * kRun) {
        gst::Pack<T, V> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = gst::load<T, V>(p + k + (u * kThreads + threadIdx.x) * V);
#pragma unroll
        for (int u = 0; u < U; ++u) add(x[u]);
    }
    if (k < n) {   // the tensor's last run, in one block
        const int64_t whole = n / V * V;
        for (int64_t q = k + (int64_t)threadIdx.x * V; q < whole; q += kThreads * V) add(gst::load<T, V>(p + q));
        if (whole + threadIdx.x < n) {
            const double d = (double)(float)p[whole + threadIdx.x];
            s = __builtin_fma(d, d, s);
        }
    }
    return s;
}

template <typename J>
__global__ __launch_bounds__(kThreads) void k_squares(J job, double* __restrict__ part)
{
    uint32_t among, blocks;
    const NormTensor& t = job.t[tensor_of_block(job, blockIdx.x, among, blocks)];
    double s = 0.0;
    auto typed = [&](auto x) {
        using T = decltype(x);
        const T* p = (const T*)t.p;
        if (t.c.apart < 0) s = squares<T>(p, t.c.n, among, blocks);
        else {
            const int64_t k0 = among * job.piece;
            each_apart(job.apart[t.c.apart], k0, min(t.c.n, k0 + job.piece),
                       [&](int64_t, int64_t at) { return p[at]; },
                       [&](int64_t, int64_t, T v) {
                           const double d = (double)(float)v;
                           s = __builtin_fma(d, d, s);
                       });
        }
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
    constexpr int V = 16 / sizeof(T);
    int64_t k = (int64_t)threadIdx.x * V;
    for (; k + V <= n; k += kThreads * V) {
        const auto x = gst::load<T, V>(p + k);
        gst::Pack<T, V> y;
#pragma unroll
        for (int e = 0; e < V; ++e) y.v[e] = gst::narrow<T>(c * (float)x.v[e]);
        gst::store_once<T, V>(o + k, y);
    }
    const int64_t t = n / V * V + threadIdx.x;
    if (t < n) o[t] = gst::narrow<T>(c * (float)p[t]);
}

// part: the norm's partials, which every block adds itself, in one order (one
// launch less, for small lists); null: the factor is in norm already.
template <typename J>
__global__ __launch_bounds__(kThreads) void k_scale(J job, const double* __restrict__ part, int64_t parts,
                                                    double max_norm, float* __restrict__ norm, int write)
{
    float c;
    if (part) {
        const double total = sqrt(total_of(part, parts));
        c = factor_of(total, max_norm);
        if (write && blockIdx.x == 0 && threadIdx.x == 0) {
            norm[0] = (float)total;
            norm[1] = c;
        }
    } else {
        c = norm[1];
    }
    uint32_t among, blocks;
    const ScaleTensor& t = job.t[tensor_of_block(job, blockIdx.x, among, blocks)];
    if (c == 1.0f && t.o == t.p) return;
    const int64_t k0 = among * job.piece, k1 = min(t.c.n, k0 + job.piece);
    auto typed = [&](auto x) {
        using T = decltype(x);
        const T* p = (const T*)t.p;
        T* o = (T*)t.o;
        if (t.c.apart < 0) scale<T>(p + k0, o + k0, k1 - k0, c);
        else
            each_apart(job.apart[t.c.apart], k0, k1, [&](int64_t, int64_t at) { return p[at]; },
                       [&](int64_t, int64_t to, T v) { o[to] = gst::narrow<T>(c * (float)v); });
    };
    if (t.c.type == GS_F32) typed(float{});
    else if (t.c.type == GS_F16) typed(gst::f16{});
    else typed(gst::bf16{});
}

// The norm of a small list, and the scaling where out tensors are given, in one
// launch of one block: its wavefronts take the list's pieces (kSmallPiece
// values) in turn, twice.
constexpr int kSmallThreads = 1024, kSmallPiece = 512;
__global__ __launch_bounds__(kSmallThreads) void k_small(ScaleJob job, double max_norm, float* __restrict__ norm,
                                                         int scaling)
{
    __shared__ double part[kSmallThreads / 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t all = job.t[job.count - 1].c.bend;
    // each(value of the type, its place, its place in out) over the wavefront's pieces
    auto pieces = [&](auto&& packs, auto&& single) {
        for (uint32_t u = wave; u < all; u += kSmallThreads / 64) {
            uint32_t among, blocks;
            const ScaleTensor& t = job.t[tensor_of_block(job, u, among, blocks)];
            const int k0 = (int)among * kSmallPiece, n = min((int)t.c.n - k0, kSmallPiece);
            auto typed = [&](auto x) {
                using T = decltype(x);
                constexpr int V = 16 / sizeof(T);
                const T* p = (const T*)t.p;
                T* o = (T*)t.o;
                if (t.c.apart >= 0) {
                    const Apart& a = job.apart[t.c.apart];
                    for (int j = lane; j < n; j += 64) {
                        const int64_t r = (uint32_t)(k0 + j) / a.cols, c = (uint32_t)(k0 + j) % a.cols;
                        single(p + r * a.stride + c, o + r * a.ostride + c);
                    }
                    return;
                }
#pragma unroll
                for (int q = 0; q < kSmallPiece; q += 64 * V) {
                    const int j = q + lane * V;
                    if (j + V <= n) packs(p + k0 + j, o + k0 + j, std::integral_constant<int, V>{});
                    else
                        for (int e = j; e < n; ++e) single(p + k0 + e, o + k0 + e);
                }
            };
            if (t.c.type == GS_F32) typed(float{});
            else if (t.c.type == GS_F16) typed(gst::f16{});
            else typed(gst::bf16{});
        }
    };
    double s = 0.0;
    auto square = [&](float x) { s = __builtin_fma((double)x, (double)x, s); };
    pieces(
        [&](const auto* p, auto*, auto v) {
            constexpr int V = decltype(v)::value;
            const auto x = gst::load<std::decay_t<decltype(*p)>, V>(p);
#pragma unroll
            for (int e = 0; e < V; ++e) square((float)x.v[e]);
        },
        [&](const auto* p, auto*) { square((float)*p); });
    s = gsd::wave_sum_d(s);
    if (lane == 0) part[wave] = s;
    __syncthreads();
    double total = 0.0;
    for (int w = 0; w < kSmallThreads / 64; ++w) total += part[w];
    total = sqrt(total);
    const float c = factor_of(total, max_norm);
    if (threadIdx.x == 0) {
        norm[0] = (float)total;
        norm[1] = c;
    }
    if (!scaling || (scaling == 2 && c == 1.0f)) return;
    pieces(
        [&](const auto* p, auto* o, auto v) {
            constexpr int V = decltype(v)::value;
            using T = std::decay_t<decltype(*p)>;
            auto x = gst::load<T, V>(p);
#pragma unroll
            for (int e = 0; e < V; ++e) x.v[e] = gst::narrow<T>(c * (float)x.v[e]);
            gst::store<T, V>(o, x);
        },
        [&](const auto* p, auto* o) { *o = gst::narrow<std::decay_t<decltype(*p)>>(c * (float)*p); });
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

// A piece, in packs of four values (p, m, v of 16 bytes each and the
// gradient's).
template <typename T>
__device__ __forceinline__ void adam(const AdamTensor& t, int64_t k0, int64_t n, float c, const AdamConst& a)
{
    constexpr int V = 4;
    float *pp = t.p + k0, *mp = t.m + k0, *vp = t.v + k0;
    const T* gp = (const T*)t.g + k0;
    for (int64_t k = (int64_t)threadIdx.x * V; k + V <= n; k += kThreads * V) {
        auto p = gst::load<float, V>(pp + k), m = gst::load<float, V>(mp + k), v = gst::load<float, V>(vp + k);
        const auto g = gst::load<T, V>(gp + k);
#pragma unroll
        for (int e = 0; e < V; ++e) adam_value(c * (float)g.v[e], p.v[e], m.v[e], v.v[e], a);
        gst::store<float, V>(pp + k, p);
        gst::store<float, V>(mp + k, m);
        gst::store<float, V>(vp + k, v);
        if (t.copy) {
            auto low = [&](auto x) {
                using O = decltype(x);
                gst::Pack<O, V> y;
#pragma unroll
                for (int e = 0; e < V; ++e) y.v[e] = gst::narrow<O>(p.v[e]);
                gst::store<O, V>((O*)t.copy + k0 + k, y);
            };
            if (t.c.type2 == GS_F32) low(float{});
            else if (t.c.type2 == GS_F16) low(gst::f16{});
            else low(gst::bf16{});
        }
    }
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

template <typename J>
__global__ __launch_bounds__(kThreads) void k_adam_list(J job, AdamConst a, const float* __restrict__ norm)
{
    float c = 1.0f;
    if (norm) {
        if (!(fabsf(norm[0]) < __builtin_inff())) return;   // not finite
        c = norm[1];
    }
    uint32_t among, blocks;
    const AdamTensor& t = job.t[tensor_of_block(job, blockIdx.x, among, blocks)];
    const int64_t k0 = among * job.piece, k1 = min(t.c.n, k0 + job.piece);
    auto typed = [&](auto x) {
        using T = decltype(x);
        if (t.c.apart < 0) adam<T>(t, k0, k1 - k0, c, a);
        else
        {
            struct Values {
                float p, m, v, g;
            };
            each_apart(job.apart[t.c.apart], k0, k1,
                       [&](int64_t k, int64_t at) {
                           return Values{t.p[k], t.m[k], t.v[k], (float)((const T*)t.g)[at]};
                       },
                       [&](int64_t k, int64_t, Values x) {
                           adam_value(c * x.g, x.p, x.m, x.v, a);
                           t.p[k] = x.p;
                           t.m[k] = x.m;
                           t.v[k] = x.v;
                           if (t.copy) put_copy(t, k, x.p);
                       });
        }
    };
    if (t.c.type == GS_F32) typed(float{});
    else if (t.c.type == GS_F16) typed(gst::f16{});
    else typed(gst::bf16{});
}

// Up to kSmall values in up to kSmallTensors tensors are one block's work.  A
// list of 5 tensors clipped: 14,000 values 6.3 us (10.6 in two launches), 28,000
// 8.2 (10.6), 42,000 11.2 (10.5); of 60 tensors and 18,000 values 14.3 (12.6).
constexpr int64_t kSmall = 32768;
constexpr int32_t kSmallTensors = 16;

// Lists of more than kLarge values are scaled in pieces of kLargePiece, after a
// launch that forms the factor; Adam takes kAdamPiece always: one or two packs
// per thread and many blocks keep the blocks that run together close together
// in memory.  354M f32: scaling 530 us with eight blocks per compute unit, 451
// with pieces of 2048; Adam with its norm 2234 us with eight blocks per compute
// unit, 2114 with pieces of 4096, 2069 with 1024.  28,000 values: 9.6 us with
// the factor formed in the scaling launch, 13.7 with a launch of its own.
constexpr int64_t kLarge = 4000000, kLargePiece = 2048, kAdamPiece = 1024;

// A list of more than kParts partials (one per tensor at least) is also scaled
// after a launch that forms the factor, as every block would add them all: of
// tensors of 40 values each, 2000 take 163 us without that launch and 166 with
// it, 3000 241 and 242, 4000 338 and 322, 100,000 45,000 and 8,430.
constexpr int64_t kParts = 3072;

// rows x cols values that lie one after the other
bool dense(const gs_tensor& t) { return t.rows <= 1 || t.stride == t.cols; }

// at least `piece` values per block, and fewer than 2^32 threads
int64_t bounded(int64_t piece, int64_t total) { return std::max(piece, ceil_div(ceil_div(total, 1 << 23), 1024) * 1024); }

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

bool is_apart(const gs_tensor* in, const gs_tensor* out, int32_t k)
{
    return !dense(in[k]) || (out && !dense(out[k]));
}

// The device table of a list that gets one (see Table), else nothing.  Taken
// apart from launch_list, so that a call has all its memory before its first
// launch writes anything.
template <typename J>
struct ListMemory {
    typename J::Tensor* t = nullptr;
    Apart* apart = nullptr;
};

template <typename J>
gs_status take_list(gs_ctx* ctx, const gs_tensor* in, const gs_tensor* out, int32_t n, std::vector<GsAlloc>* tmp,
                    ListMemory<J>* mem)
{
    typedef typename J::Tensor T;
    int64_t count = 0, aparts = 0, total = 0;
    for (int32_t k = 0; k < n; ++k)
        if (in[k].rows * in[k].cols > 0) {
            total += in[k].rows * in[k].cols;
            ++count;
            aparts += is_apart(in, out, k);
        }
    if (total <= kLarge || aparts > 0x7FFF || (count <= 3 * J::kCap && aparts <= 3 * kApart)) return GS_OK;
    mem->t = (T*)gs_malloc(ctx, sizeof(T) * count, GS_MEM_SCRATCH, tmp);
    mem->apart = (Apart*)gs_malloc(ctx, sizeof(Apart) * std::max<int64_t>(aparts, 1), GS_MEM_SCRATCH, tmp);
    return mem->t && mem->apart ? GS_OK : GS_ERR_OOM;
}

// Hands a list to a kernel: put(descriptor, tensor index) fills in the
// pointers, go(job or table, blocks) launches, once or twice.  in, out: the
// tensors whose rows may be apart (out may be null).  Allocates nothing.
template <typename J, typename P, typename G>
gs_status launch_list(gs_ctx* ctx, const gs_tensor* in, const gs_tensor* out, int32_t n, int64_t piece,
                      const ListMemory<J>& mem, P&& put, G&& go)
{
    typedef typename J::Tensor T;
    J job;
    job.piece = piece;
    job.count = job.aparts = 0;
    int64_t blocks = 0;
    int32_t at = 0, at_apart = 0;   // table entries filled
    auto flush = [&]() {
        if (job.count == 0) return;
        if (mem.t) {
            hipLaunchKernelGGL((k_fill_table<J>), dim3(1), dim3(kThreads), 0, ctx->stream, job, mem.t + at,
                               mem.apart + at_apart);
            at += job.count;
            at_apart += job.aparts;
        } else {
            go(job, (uint32_t)blocks);
            blocks = 0;
        }
        job.count = job.aparts = 0;
    };
    for (int32_t k = 0; k < n; ++k) {
        const int64_t values = in[k].rows * in[k].cols;
        if (values == 0) continue;
        const bool apart = is_apart(in, out, k);
        if (job.count == J::kCap || (apart && job.aparts == kApart)) flush();
        blocks += ceil_div(values, piece);
        T& d = job.t[job.count++];
        d.c.n = values;
        d.c.bend = (uint32_t)blocks;
        d.c.type = (int8_t)in[k].type;
        d.c.type2 = 0;
        d.c.apart = -1;
        if (apart) {
            d.c.apart = (int16_t)(at_apart + job.aparts);
            job.apart[job.aparts++] = Apart{in[k].stride, out ? out[k].stride : 0, (uint32_t)in[k].cols, 0};
        }
        put(d, k);
    }
    flush();
    if (mem.t) go(Table<T>{mem.t, mem.apart, piece, at}, (uint32_t)blocks);
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

// Tensors that are neighbouring columns of the same rows (the groups of a
// view's gradient rows) as one tensor of all those columns, so that the rows'
// cache lines are read once: neither the norm nor the scaling needs them
// apart (11 of 59 f16 columns in four tensors, 2.1M rows: 194 us, 578 with one
// tensor after the other).  in2: a second list (the outputs) that has to adjoin as well, or null.
void join_columns(const gs_tensor* in, const gs_tensor* in2, int32_t n, std::vector<gs_tensor>* out,
                  std::vector<gs_tensor>* out2)
{
    auto adjoins = [](const gs_tensor& a, const gs_tensor& b) {
        const int64_t size = a.type == GS_F32 ? 4 : 2;
        return a.type == b.type && a.rows == b.rows && a.rows > 1 && a.stride == b.stride &&
               (char*)b.data == (char*)a.data + a.cols * size && a.cols + b.cols <= a.stride && a.cols + b.cols <= 0x7FFFFFFF;
    };
    for (int32_t k = 0; k < n; ++k) {
        if (in[k].rows * in[k].cols == 0) continue;
        if (!out->empty() && adjoins(out->back(), in[k]) && (!in2 || adjoins(out2->back(), in2[k]))) {
            out->back().cols += in[k].cols;
            if (in2) out2->back().cols += in2[k].cols;
        } else {
            out->push_back(in[k]);
            if (in2) out2->push_back(in2[k]);
        }
    }
}

// the partials of a list's squares, one per block
struct Squares {
    double* part;
    int64_t parts, piece;
    ListMemory<NormJob> mem;
};

gs_status take_squares(gs_ctx* ctx, const gs_tensor* grads, int32_t n, std::vector<GsAlloc>* tmp, Squares* q)
{
    q->piece = piece_of(ctx, values(grads, n));
    q->parts = pieces(grads, n, q->piece);
    q->part = (double*)gs_malloc(ctx, 8 * std::max<int64_t>(q->parts, 1), GS_MEM_SCRATCH, tmp);
    return q->part ? take_list(ctx, grads, nullptr, n, tmp, &q->mem) : GS_ERR_OOM;
}

gs_status launch_squares(gs_ctx* ctx, const gs_tensor* grads, int32_t n, const Squares& q)
{
    GsTimerScope ts(ctx, "grad_norm");
    int64_t base = 0;
    return launch_list(ctx, grads, nullptr, n, q.piece, q.mem,
                       [&](NormTensor& d, int32_t k) { d.p = grads[k].data; },
                       [&](const auto& job, uint32_t nb) {
                           hipLaunchKernelGGL((k_squares<std::decay_t<decltype(job)>>), dim3(nb), dim3(kThreads), 0,
                                              ctx->stream, job, q.part + base);
                           base += nb;
                       });
}

}  // namespace

// k_small for lists of up to kSmall values that fit one launch: scaling 0: the
// norm alone, 1: into out, 2: in place.  False: not such a list.
static bool launch_small(gs_ctx* ctx, const gs_tensor* in, const gs_tensor* out, int32_t n, int scaling,
                         double max_norm, float* norm, gs_status* st)
{
    const int64_t total = values(in, n);
    if (total == 0 || total > kSmall || n > kSmallTensors) return false;
    static_assert(kSmallTensors <= kApart && kSmallTensors <= ScaleJob::kCap, "one launch");
    GsTimerScope ts(ctx, scaling ? "clip" : "grad_norm");
    *st = launch_list(ctx, in, out, n, kSmallPiece, ListMemory<ScaleJob>{},
                      [&](ScaleTensor& d, int32_t k) {
                          d.p = in[k].data;
                          d.o = out ? out[k].data : nullptr;
                      },
                      [&](const auto& job, uint32_t) {
                          if constexpr (std::is_same_v<std::decay_t<decltype(job)>, ScaleJob>)
                              hipLaunchKernelGGL(k_small, dim3(1), dim3(kSmallThreads), 0, ctx->stream, job, max_norm,
                                                 norm, scaling);
                      });
    return true;
}

gs_status launch_grad_norm(gs_ctx* ctx, const gs_tensor* list, int32_t count, double max_norm, float* norm,
                           std::vector<GsAlloc>* tmp)
{
    std::vector<gs_tensor> joined;
    join_columns(list, nullptr, count, &joined, nullptr);
    const gs_tensor* grads = joined.data();
    const int32_t n = (int32_t)joined.size();
    gs_status st;
    if (launch_small(ctx, grads, nullptr, n, 0, max_norm, norm, &st)) return st;
    Squares q;
    if ((st = take_squares(ctx, grads, n, tmp, &q)) != GS_OK) return st;
    if ((st = launch_squares(ctx, grads, n, q)) != GS_OK) return st;
    GsTimerScope ts(ctx, "grad_norm");
    hipLaunchKernelGGL(k_norm, dim3(1), dim3(kThreads), 0, ctx->stream, q.part, q.parts, max_norm, norm);
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

gs_status launch_clip(gs_ctx* ctx, const gs_tensor* list, int32_t count, double max_norm, const gs_tensor* to,
                      float* norm, std::vector<GsAlloc>* tmp)
{
    std::vector<gs_tensor> joined, joined_out;
    join_columns(list, to, count, &joined, &joined_out);
    const gs_tensor *in = joined.data(), *out = joined_out.data();
    const int32_t n = (int32_t)joined.size();
    const int64_t total = values(in, n);
    if (total == 0) return launch_grad_norm(ctx, in, n, max_norm, norm, tmp);
    gs_status st;
    if (launch_small(ctx, in, out, n, to == list ? 2 : 1, max_norm, norm, &st)) return st;
    Squares q;
    ListMemory<ScaleJob> mem;
    if ((st = take_squares(ctx, in, n, tmp, &q)) != GS_OK) return st;
    if ((st = take_list(ctx, in, out, n, tmp, &mem)) != GS_OK) return st;
    if ((st = launch_squares(ctx, in, n, q)) != GS_OK) return st;
    GsTimerScope ts(ctx, "clip");
    const bool large = total > kLarge, first = large || q.parts > kParts;   // the factor is formed first
    if (first)
        hipLaunchKernelGGL(k_norm, dim3(1), dim3(kThreads), 0, ctx->stream, q.part, q.parts, max_norm, norm);
    int write = 1;   // the first launch writes the norm
    return launch_list(ctx, in, out, n, large ? bounded(kLargePiece, total) : piece_of(ctx, total), mem,
                       [&](ScaleTensor& d, int32_t k) {
                           d.p = in[k].data;
                           d.o = out[k].data;
                       },
                       [&](const auto& job, uint32_t nb) {
                           hipLaunchKernelGGL((k_scale<std::decay_t<decltype(job)>>), dim3(nb), dim3(kThreads), 0,
                                              ctx->stream, job, first ? nullptr : q.part, q.parts, max_norm, norm,
                                              write);
                           write = 0;
                       });
}

gs_status launch_adam_list(gs_ctx* ctx, const gs_tensor* p, const gs_tensor* m, const gs_tensor* v, const gs_tensor* g,
                           const gs_tensor* copies, int32_t n, const gs_adam_opts* o, const float* norm,
                           std::vector<GsAlloc>* tmp)
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
    ListMemory<AdamJob> mem;
    const gs_status st = take_list(ctx, g, nullptr, n, tmp, &mem);
    if (st != GS_OK) return st;
    GsTimerScope ts(ctx, "adam_list");
    return launch_list(ctx, g, nullptr, n, bounded(kAdamPiece, values(g, n)), mem,
                       [&](AdamTensor& d, int32_t k) {
                           d.p = (float*)p[k].data;
                           d.m = (float*)m[k].data;
                           d.v = (float*)v[k].data;
                           d.g = g[k].data;
                           d.copy = copies ? copies[k].data : nullptr;
                           d.c.type2 = (int8_t)(copies ? copies[k].type : 0);
                       },
                       [&](const auto& job, uint32_t nb) {
                           hipLaunchKernelGGL((k_adam_list<std::decay_t<decltype(job)>>), dim3(nb), dim3(kThreads), 0,
                                              ctx->stream, job, a, norm);
                       });
}
