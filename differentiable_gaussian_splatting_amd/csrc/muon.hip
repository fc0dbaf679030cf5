// muon.hip -- Muon over a list of matrices: momentum, its orthogonalisation by
// Newton-Schulz products, and the update.
//
//   m = mu m + f g,  u = f g + mu m (nesterov) or m,  X = u / (|u| + 1e-7)
//   steps times: G = X X^T, P = b G + c G G, X = a X + P X
//   p = p (1 - lr wd) - lr sqrt(max(1, rows / cols)) X
// For a matrix of more rows than columns G = X^T X and X = a X + X P: the same
// with X^T, without forming it; G has the shorter side either way.
//
// The products take f32 matrices as two f16 parts (mm.h, P = 2).  The
// polynomial a s + b s^3 + c s^5 maps [0, 1.21] into itself and X starts with
// singular values of at most 1 (they are at most the Frobenius norm), so that
// |X| <= 1.21, |G| <= 1.47 and |P| <= 2.81 (the largest |b t + c t^2| for t up
// to 1.47): scaled by 2^15, 2^15 and 2^14 all stay below 65504, and a value is
// held to 2^-22 of itself down to 2^-18 of those bounds.  Products in one bf16
// part each would lose 2^-9 of X per step, and the polynomial multiplies what
// the first steps lose by up to a^5 = 485.
#include <algorithm>
#include <cmath>

#include "gs_internal.h"
#include "gs_tensor.h"
#include "mm.h"

namespace {

using namespace gsm;

typedef gst::Pack<float, 4> Four;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr double kEps = 1e-7;
constexpr float kScaleX = 32768.0f, kScaleP = 16384.0f;   // of X and G, and of P

constexpr int kThreads = 256;
constexpr int kPiece = 4096;      // values of a block of the elementwise kernels
constexpr int kGroup = 40;        // matrices of a launch (kernel arguments within 4 KB)

// A matrix of a group.  Its X, G and P start at x, s and s in the group's
// workspaces.
struct Matrix {
    float *p, *m;
    const void* g;
    void* copy;
    int64_t gld;
    int64_t x, s;
    int32_t rows, cols;
    uint32_t piece_end;           // pieces of the matrices up to this one
    int8_t gtype, ctype;
};
struct Job {
    Matrix t[kGroup];
    int32_t count;
};
struct MuonConst {
    float mu, lr, keep;           // keep = 1 - lr weight_decay
    int32_t nesterov;
};

struct Shape {
    int64_t x, s;
    int32_t rows, cols;
    uint32_t tile_end;            // tiles of the matrices up to this one
};
struct MmJob {
    Shape t[kGroup];
    int32_t count;
};
static_assert(sizeof(Job) <= 3840 && sizeof(MmJob) <= 3840, "kernel arguments");

// the matrix that holds piece (tile) b, and the pieces before it
template <typename J, typename F>
__device__ __forceinline__ int matrix_of(const J& job, uint32_t b, F end, uint32_t& before)
{
    int lo = 0, hi = job.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (b < end(job.t[mid])) hi = mid;
        else lo = mid + 1;
    }
    before = lo ? end(job.t[lo - 1]) : 0u;
    return lo;
}

template <typename F>
__device__ __forceinline__ void with_type_device(int type, F&& f)
{
    if (type == GS_F32) f(float{});
    else if (type == GS_F16) f(gst::f16{});
    else f(gst::bf16{});
}

__device__ __forceinline__ float gradient(const Matrix& t, int64_t at)
{
    const int64_t r = at / t.cols, c = at - r * t.cols;
    float x = 0.0f;
    with_type_device(t.gtype, [&](auto s) { x = (float)((const decltype(s)*)t.g)[r * t.gld + c]; });
    return x;
}

__device__ __forceinline__ double block_sum(double x, double* part)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

// momentum, and the squares of u (f64, one partial per piece)
__global__ __launch_bounds__(kThreads) void k_momentum(const Job job, const MuonConst o, const float* __restrict__ norm,
                                                       double* __restrict__ part)
{
    __shared__ double sums[4];
    if (norm && !isfinite(norm[0])) return;
    const float f = norm ? norm[1] : 1.0f;
    uint32_t before;
    const Matrix& t = job.t[matrix_of(job, blockIdx.x, [](const Matrix& q) { return q.piece_end; }, before)];
    const int64_t n = (int64_t)t.rows * t.cols, at = (int64_t)(blockIdx.x - before) * kPiece;
    double sum = 0.0;
    for (int64_t i = at + threadIdx.x; i < min(n, at + kPiece); i += kThreads) {
        const float g = f * gradient(t, i), m = o.mu * t.m[i] + g;
        t.m[i] = m;
        const float u = o.nesterov ? g + o.mu * m : m;
        sum += (double)u * u;
    }
    sum = block_sum(sum, sums);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// X = u / (|u| + eps)
__global__ __launch_bounds__(kThreads) void k_start(const Job job, const MuonConst o, const float* __restrict__ norm,
                                                    const double* __restrict__ part, float* __restrict__ x)
{
    __shared__ double sums[4];
    if (norm && !isfinite(norm[0])) return;
    const float f = norm ? norm[1] : 1.0f;
    uint32_t before;
    const Matrix& t = job.t[matrix_of(job, blockIdx.x, [](const Matrix& q) { return q.piece_end; }, before)];
    const int64_t n = (int64_t)t.rows * t.cols, at = (int64_t)(blockIdx.x - before) * kPiece;
    double sum = 0.0;
    for (uint32_t b = before + threadIdx.x; b < t.piece_end; b += kThreads) sum += part[b];
    const float inv = (float)(1.0 / (sqrt(block_sum(sum, sums)) + kEps));
    for (int64_t i = at + threadIdx.x; i < min(n, at + kPiece); i += kThreads) {
        const float m = t.m[i];
        x[t.x + i] = (o.nesterov ? f * gradient(t, i) + o.mu * m : m) * inv;
    }
}

// parameters and their copies
__global__ __launch_bounds__(kThreads) void k_apply(const Job job, const MuonConst o, const float* __restrict__ norm,
                                                    const float* __restrict__ x)
{
    if (norm && !isfinite(norm[0])) return;
    uint32_t before;
    const Matrix& t = job.t[matrix_of(job, blockIdx.x, [](const Matrix& q) { return q.piece_end; }, before)];
    const int64_t n = (int64_t)t.rows * t.cols, at = (int64_t)(blockIdx.x - before) * kPiece;
    const float rate = o.lr * sqrtf(fmaxf(1.0f, (float)t.rows / (float)t.cols));
    for (int64_t i = at + threadIdx.x; i < min(n, at + kPiece); i += kThreads) {
        const float p = t.p[i] * o.keep - rate * x[t.x + i];
        t.p[i] = p;
        if (t.copy) with_type_device(t.ctype, [&](auto s) { ((decltype(s)*)t.copy)[i] = gst::narrow<decltype(s)>(p); });
    }
}

enum { kGram, kPoly, kNext };

// One tile of a matrix's product: G (kGram), P from G (kPoly) or the next X.
// G and P are symmetric: their tiles on and below the diagonal are computed and
// those below it written to both places.
template <int KIND, bool TALL, typename T>
__global__ __launch_bounds__(T::NT, 2) void k_newton(const MmJob job, const float* __restrict__ from, float* __restrict__ to,
                                                  const float* __restrict__ poly)
{
    constexpr bool ACOL = KIND == kGram && TALL, BCOL = ACOL || (KIND == kNext && !TALL);
    __shared__ Lds<float, 2, T> lds;
    const uint32_t b = (uint32_t)xcd_order(blockIdx.x, gridDim.x);
    uint32_t before;
    const Shape t = job.t[matrix_of(job, b, [](const Shape& q) { return q.tile_end; }, before)];
    const int64_t side = TALL ? t.cols : t.rows, length = TALL ? t.rows : t.cols;
    const int64_t m = KIND == kNext ? t.rows : side, n = KIND == kNext ? t.cols : side;
    const int64_t k = KIND == kGram ? length : side;
    int64_t i, j;
    if constexpr (KIND == kNext) {
        tile_at(b - before, (m + T::BM - 1) / T::BM, (n + T::BN - 1) / T::BN, i, j);
    } else {
        static_assert(T::BM == T::BN, "square tiles");
        const int t = (int)(b - before);
        int r = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
        while (r * (r + 1) / 2 > t) --r;
        while ((r + 1) * (r + 2) / 2 <= t) ++r;
        i = r;
        j = t - r * (r + 1) / 2;
    }
    const float* src = from + (KIND == kPoly ? t.s : t.x);
    const Operand x = {src, KIND == kPoly ? side : t.cols, KIND == kPoly ? side : KIND == kGram ? side : TALL ? m : n,
                       kScaleX, 0};
    Operand a = x, bo = x;
    if constexpr (KIND == kNext) (TALL ? bo : a) = Operand{poly + t.s, side, side, kScaleP, 0};
    f32x4 acc[T::NI][T::MI];
#pragma unroll
    for (int q = 0; q < T::NI; ++q)
#pragma unroll
        for (int r = 0; r < T::MI; ++r) acc[q][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    mm_tile<float, 2, ACOL, BCOL, T>(a, bo, i * T::BM, j * T::BN, 0, k, lds, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t mw = i * T::BM + (wave % T::WM) * T::MI * 16 + (lane & 15);
    const int64_t nw = j * T::BN + (wave / T::WM) * T::NI * 16 + (lane >> 4) * 4;
    const float down = 1.0f / kScaleX / (KIND == kNext ? kScaleP : kScaleX);
    float* dst = to + (KIND == kNext ? t.x : t.s);
#pragma unroll
    for (int r = 0; r < T::MI; ++r) {
        const int64_t row = mw + r * 16;
        if (row >= m) continue;
#pragma unroll
        for (int q = 0; q < T::NI; ++q) {
            const int64_t col = nw + q * 16, at = row * n + col;
            if (col >= n) continue;
            const int valid = (int)min((int64_t)4, n - col);
            f32x4 y = acc[q][r] * down, old = y;
            if constexpr (KIND != kGram) {
                if (valid == 4) {
                    old = __builtin_bit_cast(f32x4, gst::load<float, 4>(src + at));
                } else {
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        if (w < valid) old[w] = src[at + w];
                }
                y = KIND == kPoly ? kC * y + kB * old : y + kA * old;
            }
            if (valid == 4) {
                gst::store<float, 4>(dst + at, __builtin_bit_cast(Four, y));
            } else {
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (w < valid) dst[at + w] = y[w];
            }
            if (KIND != kNext && i != j) {
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (w < valid) dst[(col + w) * n + row] = y[w];
            }
        }
    }
}

typedef Tile<256, 256, 32, 2, 4, 2> Large;
typedef Tile<128, 128, 32, 2, 2, 1> Medium;
typedef Tile<64, 64, 32, 2, 2, 2> Small;
typedef Tile<64, 64, 32, 2, 2, 2, true> Tiny;

// tiles of a matrix's product
template <int KIND>
int64_t tiles_of(const Matrix& t, int bm, int bn)
{
    const int64_t side = std::min(t.rows, t.cols), s = ceil_div(side, bm);
    return KIND == kNext ? ceil_div(t.rows, bm) * ceil_div(t.cols, bn) : s * (s + 1) / 2;
}

template <int KIND, bool TALL, typename T>
void launch_tiles(gs_ctx* ctx, const Job& job, const float* from, float* to, const float* poly)
{
    MmJob mm{};
    uint32_t tiles = 0;
    for (int32_t k = 0; k < job.count; ++k) {
        const Matrix& t = job.t[k];
        tiles += (uint32_t)tiles_of<KIND>(t, T::BM, T::BN);
        mm.t[mm.count++] = Shape{t.x, t.s, t.rows, t.cols, tiles};
    }
    hipLaunchKernelGGL((k_newton<KIND, TALL, T>), dim3(tiles), dim3(T::NT), 0, ctx->stream, mm, from, to, poly);
}

// What a group's product takes with a tile of which per_cu blocks run on a
// compute unit, each in step_us for 32 values of k (large matrices: 256 x 256
// at 345 TFLOP/s, 128 x 128 at 295).
template <int KIND, typename T>
double cost_us(const gs_ctx* ctx, const Job& job, int per_cu, double step_us)
{
    int64_t work = 0, longest = 0, tiles = 0;
    for (int32_t k = 0; k < job.count; ++k) {
        const Matrix& t = job.t[k];
        const int64_t steps = ceil_div(KIND == kGram ? std::max(t.rows, t.cols) : std::min(t.rows, t.cols), T::BK);
        const int64_t n = tiles_of<KIND>(t, T::BM, T::BN);
        tiles += n;
        work += n * steps;
        longest = std::max(longest, steps);
    }
    const double rounds = (double)ceil_div(tiles, (int64_t)per_cu * ctx->num_cu);
    return rounds * std::max((double)work / (double)tiles, (double)longest / rounds) * step_us;
}

template <int KIND, bool TALL>
void launch_newton(gs_ctx* ctx, const Job& job, bool tiny, const float* from, float* to, const float* poly)
{
    if (tiny) return launch_tiles<KIND, TALL, Tiny>(ctx, job, from, to, poly);
    const double large = cost_us<KIND, Large>(ctx, job, 1, 3.1), medium = cost_us<KIND, Medium>(ctx, job, 2, 1.8),
                 small = cost_us<KIND, Small>(ctx, job, 3, 0.9);
    if (large <= medium && large <= small) launch_tiles<KIND, TALL, Large>(ctx, job, from, to, poly);
    else if (medium <= small) launch_tiles<KIND, TALL, Medium>(ctx, job, from, to, poly);
    else launch_tiles<KIND, TALL, Small>(ctx, job, from, to, poly);
}

template <bool TALL>
void newton_schulz(gs_ctx* ctx, const Job& job, bool tiny, int steps, float** x, float** other, float* gram, float* poly)
{
    for (int s = 0; s < steps; ++s) {
        launch_newton<kGram, TALL>(ctx, job, tiny, *x, gram, nullptr);
        launch_newton<kPoly, TALL>(ctx, job, tiny, gram, poly, nullptr);
        launch_newton<kNext, TALL>(ctx, job, tiny, *x, *other, poly);
        std::swap(*x, *other);
    }
}

// the matrices whose products share launches, and the floats of their X and G
struct Group {
    Job job;
    int64_t x, s;
    uint32_t pieces;
    bool tall, tiny;              // more rows than columns; a side below 8 (Stage in mm.h)
};
constexpr int64_t kGroupValues = 1 << 27;   // of X: one 512 MB workspace, of which a step needs four

}  // namespace

gs_status launch_muon_list(gs_ctx* ctx, const gs_tensor* p, const gs_tensor* m, const gs_tensor* g,
                           const gs_tensor* copies, int32_t n, const gs_muon_opts* o, const float* norm,
                           std::vector<GsAlloc>* tmp)
{
    const MuonConst c = {(float)o->momentum, (float)o->lr, (float)(1.0 - o->lr * o->weight_decay), o->nesterov};
    std::vector<Group> groups;
    int64_t x = 0, s = 0, pieces = 0;
    for (int kind = 0; kind < 4; ++kind) {
        const bool tall = kind & 1, tiny = kind & 2;
        bool open = false;
        for (int32_t k = 0; k < n; ++k) {
            const int64_t rows = p[k].rows, cols = p[k].cols, values = rows * cols, side = std::min(rows, cols);
            if (values == 0 || (rows > cols) != tall || (side < 8) != tiny) continue;
            if (open && (groups.back().job.count == kGroup || groups.back().x + values > kGroupValues)) open = false;
            if (!open) {
                groups.push_back(Group{});
                groups.back().tall = tall;
                groups.back().tiny = tiny;
                open = true;
            }
            Group& q = groups.back();
            q.pieces += (uint32_t)ceil_div(values, kPiece);
            q.job.t[q.job.count++] = Matrix{(float*)p[k].data, (float*)m[k].data, g[k].data,
                                            copies ? copies[k].data : nullptr, g[k].stride, q.x, q.s, (int32_t)rows,
                                            (int32_t)cols, q.pieces, (int8_t)g[k].type,
                                            (int8_t)(copies ? copies[k].type : 0)};
            q.x += ceil_div(values, 64) * 64;   // each matrix starts on a cache line
            q.s += ceil_div(side * side, 64) * 64;
            x = std::max(x, q.x);
            s = std::max(s, q.s);
            pieces = std::max<int64_t>(pieces, q.pieces);
        }
    }
    if (groups.empty()) return GS_OK;
    double* part = (double*)gs_malloc(ctx, 8 * pieces, GS_MEM_SCRATCH, tmp);
    float* xs = (float*)gs_malloc(ctx, 4 * 2 * x, GS_MEM_SCRATCH, tmp);
    float* ss = (float*)gs_malloc(ctx, 4 * 2 * s, GS_MEM_SCRATCH, tmp);
    if (!part || !xs || !ss) return GS_ERR_OOM;
    for (const Group& q : groups) {
        GsTimerScope ts(ctx, "muon");
        float *now = xs, *other = xs + x;
        const dim3 grid(q.pieces), block(kThreads);
        hipLaunchKernelGGL(k_momentum, grid, block, 0, ctx->stream, q.job, c, norm, part);
        hipLaunchKernelGGL(k_start, grid, block, 0, ctx->stream, q.job, c, norm, part, now);
        if (q.tall) newton_schulz<true>(ctx, q.job, q.tiny, o->steps, &now, &other, ss, ss + s);
        else newton_schulz<false>(ctx, q.job, q.tiny, o->steps, &now, &other, ss, ss + s);
        hipLaunchKernelGGL(k_apply, grid, block, 0, ctx->stream, q.job, c, norm, now);
        GS_HIP(ctx, hipGetLastError());
    }
    return GS_OK;
}
