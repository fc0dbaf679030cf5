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

// floats from a row of X, G or P to the next
__host__ __device__ constexpr int64_t padded(int64_t cols) { return (cols + 31) / 32 * 32; }

constexpr int kThreads = 256;
constexpr int kPiece = 4096;      // values of a block of the elementwise kernels
constexpr int kGroup = 40;        // matrices of a launch (kernel arguments within 4 KB)

// A matrix of a group.  Its X, G and P start at x, s and s in the group's
// workspaces; their rows start on cache lines (padded).
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

__device__ __forceinline__ float gradient(const Matrix& t, int64_t r, int64_t c)
{
    float x = 0.0f;
    with_type_device(t.gtype, [&](auto s) { x = (float)((const decltype(s)*)t.g)[r * t.gld + c]; });
    return x;
}

// The calling thread's values of a piece: f(flat index, row, column).
template <typename F>
__device__ __forceinline__ void each_value(const Matrix& t, uint32_t piece, F&& f)
{
    const int64_t first = (int64_t)piece * kPiece, end = min((int64_t)t.rows * t.cols, first + kPiece);
    const int32_t down = kThreads / t.cols, along = kThreads % t.cols;
    int64_t i = first + threadIdx.x, r = i / t.cols;
    int32_t c = (int32_t)(i - r * t.cols);
#pragma unroll 4
    for (; i < end; i += kThreads) {
        f(i, r, c);
        r += down;
        c += along;
        if (c >= t.cols) {
            c -= t.cols;
            ++r;
        }
    }
}

// sum over a block of W waves, in a fixed order
template <int W>
__device__ __forceinline__ double block_sum(double x, double* part)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) x += part[w];
    return x;
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
    double sum = 0.0;
    each_value(t, blockIdx.x - before, [&](int64_t i, int64_t r, int32_t c) {
        const float g = f * gradient(t, r, c), m = o.mu * t.m[i] + g;
        t.m[i] = m;
        const float u = o.nesterov ? g + o.mu * m : m;
        sum += (double)u * u;
    });
    sum = block_sum<4>(sum, sums);
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
    double sum = 0.0;
    for (uint32_t b = before + threadIdx.x; b < t.piece_end; b += kThreads) sum += part[b];
    const float inv = (float)(1.0 / (sqrt(block_sum<4>(sum, sums)) + kEps));
    const int64_t ld = padded(t.cols);
    each_value(t, blockIdx.x - before, [&](int64_t i, int64_t r, int32_t c) {
        const float m = t.m[i];
        x[t.x + r * ld + c] = (o.nesterov ? f * gradient(t, r, c) + o.mu * m : m) * inv;
    });
}

__device__ __forceinline__ float update_rate(const MuonConst& o, int32_t rows, int32_t cols)
{
    return o.lr * sqrtf(fmaxf(1.0f, (float)rows / (float)cols));
}

__device__ __forceinline__ void write_parameter(const Matrix& t, int64_t i, float p)
{
    t.p[i] = p;
    if (t.copy) with_type_device(t.ctype, [&](auto s) { ((decltype(s)*)t.copy)[i] = gst::narrow<decltype(s)>(p); });
}

// parameters and their copies
__global__ __launch_bounds__(kThreads) void k_apply(const Job job, const MuonConst o, const float* __restrict__ norm,
                                                    const float* __restrict__ x)
{
    if (norm && !isfinite(norm[0])) return;
    uint32_t before;
    const Matrix& t = job.t[matrix_of(job, blockIdx.x, [](const Matrix& q) { return q.piece_end; }, before)];
    const float rate = update_rate(o, t.rows, t.cols);
    const int64_t ld = padded(t.cols);
    each_value(t, blockIdx.x - before, [&](int64_t i, int64_t r, int32_t c) {
        write_parameter(t, i, t.p[i] * o.keep - rate * x[t.x + r * ld + c]);
    });
}

enum { kGram, kPoly, kNext };

// One tile of a matrix's product: G (kGram), P from G (kPoly) or the next X.
// G and P are symmetric: their tiles on and below the diagonal are computed and
// those below it written to both places.
template <int KIND, bool TALL, typename T>
__global__ __launch_bounds__(T::NT, 2) void k_newton(const MmJob job, const float* __restrict__ from, float* __restrict__ to,
                                                  const float* __restrict__ poly, int splits, int64_t split_size)
{
    constexpr bool ACOL = KIND == kGram && TALL, BCOL = ACOL || (KIND == kNext && !TALL);
    __shared__ Lds<float, 2, T> lds;
    uint32_t b = (uint32_t)xcd_order(blockIdx.x, gridDim.x), before;
    const uint32_t tiles = gridDim.x / (uint32_t)splits, split = KIND == kGram ? b / tiles : 0;
    if constexpr (KIND == kGram) b -= split * tiles;
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
    const int64_t lds_ = padded(side), ldx = padded(t.cols);   // of G and P, of X
    const Operand x = {src, KIND == kPoly ? lds_ : ldx, KIND == kPoly ? side : KIND == kGram ? side : TALL ? m : n,
                       kScaleX, 0};
    Operand a = x, bo = x;
    if constexpr (KIND == kNext) (TALL ? bo : a) = Operand{poly + t.s, lds_, side, kScaleP, 0};
    f32x4 acc[T::NI][T::MI];
#pragma unroll
    for (int q = 0; q < T::NI; ++q)
#pragma unroll
        for (int r = 0; r < T::MI; ++r) acc[q][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    int64_t k0 = 0, k1 = k;
    if constexpr (KIND == kGram) {
        const int64_t each = ((k + T::BK - 1) / T::BK + splits - 1) / splits * T::BK;
        k0 = min(k, split * each);
        k1 = min(k, k0 + each);
    }
    mm_tile<float, 2, ACOL, BCOL, T>(a, bo, i * T::BM, j * T::BN, k0, k1, lds, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t mw = i * T::BM + (wave % T::WM) * T::MI * 16 + (lane & 15);
    const int64_t nw = j * T::BN + (wave / T::WM) * T::NI * 16 + (lane >> 4) * 4;
    const float down = 1.0f / kScaleX / (KIND == kNext ? kScaleP : kScaleX);
    float* dst = to + (KIND == kNext ? t.x : t.s) + (KIND == kGram ? split * split_size : 0);
    const int64_t ld = KIND == kNext ? ldx : lds_;
#pragma unroll
    for (int r = 0; r < T::MI; ++r) {
        const int64_t row = mw + r * 16;
        if (row >= m) continue;
#pragma unroll
        for (int q = 0; q < T::NI; ++q) {
            const int64_t col = nw + q * 16, at = row * ld + col;
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
                    if (w < valid) dst[(col + w) * ld + row] = y[w];
            }
        }
    }
}

// G = sum of its splits, over all of a group's G
__global__ __launch_bounds__(kThreads) void k_sum_splits(float* __restrict__ g, int64_t n, int splits)
{
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * kThreads * 4) {
        f32x4 x = *reinterpret_cast<const f32x4*>(g + i);
        for (int s = 1; s < splits; ++s) x += *reinterpret_cast<const f32x4*>(g + s * n + i);
        *reinterpret_cast<f32x4*>(g + i) = x;
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

// the matrices whose products share launches, and the floats of their X and G
struct Group {
    Job job;
    int64_t x, s;
    uint32_t pieces;
    bool tall, tiny;              // more rows than columns; a side below 8 (Stage in mm.h)
    int splits;                   // of G's products
};

template <int KIND, bool TALL, typename T>
void launch_tiles(gs_ctx* ctx, const Group& q, const float* from, float* to, const float* poly)
{
    const int splits = KIND == kGram ? q.splits : 1;
    MmJob mm{};
    uint32_t tiles = 0;
    for (int32_t k = 0; k < q.job.count; ++k) {
        const Matrix& t = q.job.t[k];
        tiles += (uint32_t)tiles_of<KIND>(t, T::BM, T::BN);
        mm.t[mm.count++] = Shape{t.x, t.s, t.rows, t.cols, tiles};
    }
    hipLaunchKernelGGL((k_newton<KIND, TALL, T>), dim3(tiles * splits), dim3(T::NT), 0, ctx->stream, mm, from, to, poly,
                       splits, q.s);
    if (splits > 1)
        hipLaunchKernelGGL(k_sum_splits, dim3((uint32_t)std::min<int64_t>(ceil_div(q.s, 4 * kThreads), 2048)),
                           dim3(kThreads), 0, ctx->stream, to, q.s, splits);
}

// What a group's product takes with a tile: for a step of 32 values of k,
// once us for every round of `resident` tiles on each compute unit and each us
// for every tile (measured: 128 x 128 takes 1.3 and 2.0 us for one and two a
// unit, 64 x 64 0.9, 1.5 and 3.1 for two, four and eight, 256 x 256 3.1).
template <int KIND, typename T>
double cost_us(const gs_ctx* ctx, const Job& job, int splits, int resident, double once, double each)
{
    int64_t work = 0, longest = 0, tiles = 0;
    for (int32_t k = 0; k < job.count; ++k) {
        const Matrix& t = job.t[k];
        const int64_t steps = ceil_div(ceil_div(KIND == kGram ? std::max(t.rows, t.cols) : std::min(t.rows, t.cols), T::BK), splits);
        const int64_t n = tiles_of<KIND>(t, T::BM, T::BN) * splits;
        tiles += n;
        work += n * (steps + 1);
        longest = std::max(longest, steps + 1);
    }
    const int64_t rounds = ceil_div(tiles, (int64_t)resident * ctx->num_cu), on_each = ceil_div(tiles, ctx->num_cu);
    return std::max((double)work / (double)tiles * ((double)rounds * once + (double)on_each * each),
                    (double)longest * (once + each));
}

// the cheapest tile, and its cost
template <int KIND>
int choose_tile(const gs_ctx* ctx, const Job& job, int splits, double* us)
{
    const double cost[3] = {cost_us<KIND, Large>(ctx, job, splits, 1, 0.1, 3.0),
                            cost_us<KIND, Medium>(ctx, job, splits, 2, 0.5, 0.75),
                            cost_us<KIND, Small>(ctx, job, splits, 5, 0.25, 0.33)};
    int best = 0;
    for (int k = 1; k < 3; ++k)
        if (cost[k] < cost[best]) best = k;
    *us = cost[best];
    return best;
}

template <int KIND, bool TALL>
void launch_newton(gs_ctx* ctx, const Group& q, const float* from, float* to, const float* poly)
{
    double us;
    const int tile = choose_tile<KIND>(ctx, q.job, KIND == kGram ? q.splits : 1, &us);
    if (q.tiny) launch_tiles<KIND, TALL, Tiny>(ctx, q, from, to, poly);
    else if (tile == 0) launch_tiles<KIND, TALL, Large>(ctx, q, from, to, poly);
    else if (tile == 1) launch_tiles<KIND, TALL, Medium>(ctx, q, from, to, poly);
    else launch_tiles<KIND, TALL, Small>(ctx, q, from, to, poly);
}

// How often G's product is split over its long k: few tiles, a few matrices of
// one long side each, leave the card idle otherwise.
int choose_splits(const gs_ctx* ctx, const Group& q)
{
    int best = 1;
    double least = 0.0;
    for (int s = 1; s <= 32; s *= 2) {
        if (s > 1 && s * q.s > (1ll << 26)) break;
        double us;
        choose_tile<kGram>(ctx, q.job, s, &us);
        if (s > 1) us += 5.0 + 4.0 * (s + 1) * q.s / 3e6;   // the sums' launch and bytes
        if (s > 1 && us >= least) continue;
        least = us;
        best = s;
    }
    return best;
}

template <bool TALL>
void newton_schulz(gs_ctx* ctx, const Group& q, int steps, float** x, float** other, float* gram, float* poly)
{
    for (int s = 0; s < steps; ++s) {
        launch_newton<kGram, TALL>(ctx, q, *x, gram, nullptr);
        launch_newton<kPoly, TALL>(ctx, q, gram, poly, nullptr);
        launch_newton<kNext, TALL>(ctx, q, *x, *other, poly);
        std::swap(*x, *other);
    }
}

constexpr int64_t kGroupValues = 1 << 27;   // of X: one 512 MB workspace, of which a step needs four

// ---- small matrices ---------------------------------------------------------

// A matrix that fits one block: the whole update in one launch.  With S and L
// the shorter and the longer side, rounded up to 32, each of the block's W
// waves owns a 32 x 32 block of G (and P) and one of X, in registers, in f32;
// the products read them from LDS, as f16 pairs in rows of L + 8 and S + 8
// values (the 16 bytes spread the rows over the banks).  A tall matrix is
// loaded turned round.
template <int W>
struct SmallLds {
    static constexpr int kBlock = 32 * 32 * W;                       // values of X at most
    static constexpr int kG = W == 16 ? 128 : 64;                    // S at most
    f16 x[2][kBlock + 8 * kG];
    f16 g[2][kG * (kG + 8)];
    double sums[W];
};
template <int W>
constexpr bool fits(int64_t rows, int64_t cols)
{
    const int64_t s = padded(std::min(rows, cols)), l = padded(std::max(rows, cols));
    return s <= SmallLds<W>::kG && s * l <= SmallLds<W>::kBlock;
}

__device__ __forceinline__ void put_pair(f16* hi, f16* lo, f32x4 v, float scale)
{
    gst::Pack<f16, 4> h, l;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float x = v[j] * scale;
        h.v[j] = (f16)x;
        l.v[j] = (f16)(x - (float)h.v[j]);
    }
    *reinterpret_cast<gst::Pack<f16, 4>*>(__builtin_assume_aligned(hi, 8)) = h;
    *reinterpret_cast<gst::Pack<f16, 4>*>(__builtin_assume_aligned(lo, 8)) = l;
}

// 16 rows from r on of a row operand at k: a lane's 8 values
__device__ __forceinline__ gst::Pack<f16, 8> row_part(const f16* p, int ld, int r, int k, int lane)
{
    return *reinterpret_cast<const gst::Pack<f16, 8>*>(
        __builtin_assume_aligned(p + (r + (lane & 15)) * ld + k + (lane >> 4) * 8, 16));
}
// 16 columns from c on at k of an operand whose k runs down the columns
__device__ __forceinline__ gst::Pack<f16, 8> col_part(const f16* p, int ld, int c, int k, int lane)
{
    typedef short v4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4* at;
    const f16* q = p + (k + (lane >> 4) * 8 + ((lane >> 2) & 3)) * ld + c + (lane & 3) * 4;
    const v4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at)q);
    const v4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((at)(q + 4 * ld));
    gst::Pack<f16, 8> both;
    __builtin_memcpy(&both.v[0], &lo, 8);
    __builtin_memcpy(&both.v[4], &hi, 8);
    return both;
}

// acc[i][j] += the 32 x 32 block with rows from m on (j) and columns from n on
// (i): a of the rows, b of the columns, both over k values
template <bool BCOL>
__device__ __forceinline__ void block_product(const f16* ah, const f16* al, int lda, int m, const f16* bh, const f16* bl,
                                              int ldb, int n, int k, int lane, f32x4 (&acc)[2][2])
{
    for (int at = 0; at < k; at += 32) {
        gst::Pack<f16, 8> a[2][2], b[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a[0][i] = row_part(ah, lda, m + i * 16, at, lane);
            a[1][i] = row_part(al, lda, m + i * 16, at, lane);
            b[0][i] = BCOL ? col_part(bh, ldb, n + i * 16, at, lane) : row_part(bh, ldb, n + i * 16, at, lane);
            b[1][i] = BCOL ? col_part(bl, ldb, n + i * 16, at, lane) : row_part(bl, ldb, n + i * 16, at, lane);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                acc[i][j] = mfma(b[1][i], a[0][j], acc[i][j]);
                acc[i][j] = mfma(b[0][i], a[1][j], acc[i][j]);
                acc[i][j] = mfma(b[0][i], a[0][j], acc[i][j]);
            }
    }
}

template <int W>
__global__ __launch_bounds__(W * 64) void k_small(const Job job, const MuonConst o, const float* __restrict__ norm,
                                                  int steps)
{
    __shared__ __align__(16) SmallLds<W> lds;
    if (norm && !isfinite(norm[0])) return;
    const float f = norm ? norm[1] : 1.0f;
    const Matrix& t = job.t[blockIdx.x];
    const bool tall = t.rows > t.cols;
    const int s = tall ? t.cols : t.rows, l = tall ? t.rows : t.cols;
    const int S = (int)padded(s), L = (int)padded(l), ldx = L + 8, ldg = S + 8;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // the wave's blocks: row and column of X, and of G
    const int xm = wave % (S / 32) * 32, xn = wave / (S / 32) * 32, gm = xm, gn = xn;
    const bool has_x = xn < L, has_g = gn < S;
    const int dm = lane & 15, dn = (lane >> 4) * 4;   // the lane's place in a 16 x 16 result
    f32x4 x[2][2], g[2][2];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[i][j] = g[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            const int r = xm + j * 16 + dm;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int c = xn + i * 16 + dn + w;
                if (!has_x || r >= s || c >= l) continue;
                const int64_t row = tall ? c : r, col = tall ? r : c, at = row * t.cols + col;
                const float grad = f * gradient(t, row, col), m = o.mu * t.m[at] + grad;
                t.m[at] = m;
                const float u = o.nesterov ? grad + o.mu * m : m;
                x[i][j][w] = u;
                sum += (double)u * u;
            }
        }
    const float inv = (float)(1.0 / (sqrt(block_sum<W>(sum, lds.sums)) + kEps));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) x[i][j] *= inv;
    const float down = 1.0f / kScaleX / kScaleX;
    for (int step = 0; step < steps; ++step) {
        f32x4 acc[2][2];
        auto clear = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        };
        auto put = [&](f16* hi, f16* lo, int ld, int m, int n, f32x4 (&v)[2][2], float scale) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int at = (m + j * 16 + dm) * ld + n + i * 16 + dn;
                    put_pair(hi + at, lo + at, v[i][j], scale);
                }
        };
        if (has_x) put(lds.x[0], lds.x[1], ldx, xm, xn, x, kScaleX);
        __syncthreads();
        if (has_g) {
            clear();
            block_product<false>(lds.x[0], lds.x[1], ldx, gm, lds.x[0], lds.x[1], ldx, gn, L, lane, acc);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) g[i][j] = acc[i][j] * down;
            put(lds.g[0], lds.g[1], ldg, gm, gn, g, kScaleX);
        }
        __syncthreads();
        if (has_g) {
            clear();
            block_product<false>(lds.g[0], lds.g[1], ldg, gm, lds.g[0], lds.g[1], ldg, gn, S, lane, acc);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) g[i][j] = kC * (acc[i][j] * down) + kB * g[i][j];
        }
        __syncthreads();
        if (has_g) put(lds.g[0], lds.g[1], ldg, gm, gn, g, kScaleP);
        __syncthreads();
        if (has_x) {
            clear();
            block_product<true>(lds.g[0], lds.g[1], ldg, xm, lds.x[0], lds.x[1], ldx, xn, S, lane, acc);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) x[i][j] = acc[i][j] * (1.0f / kScaleX / kScaleP) + kA * x[i][j];
        }
        __syncthreads();
    }
    const float rate = update_rate(o, t.rows, t.cols);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = xm + j * 16 + dm;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int c = xn + i * 16 + dn + w;
                if (!has_x || r >= s || c >= l) continue;
                const int64_t at = tall ? (int64_t)c * t.cols + r : (int64_t)r * t.cols + c;
                write_parameter(t, at, t.p[at] * o.keep - rate * x[i][j][w]);
            }
        }
}

}  // namespace

gs_status launch_muon_list(gs_ctx* ctx, const gs_tensor* p, const gs_tensor* m, const gs_tensor* g,
                           const gs_tensor* copies, int32_t n, const gs_muon_opts* o, const float* norm,
                           std::vector<GsAlloc>* tmp)
{
    const MuonConst c = {(float)o->momentum, (float)o->lr, (float)(1.0 - o->lr * o->weight_decay), o->nesterov};
    const auto describe = [&](int32_t k) {
        return Matrix{(float*)p[k].data, (float*)m[k].data, g[k].data, copies ? copies[k].data : nullptr, g[k].stride, 0, 0,
                      (int32_t)p[k].rows, (int32_t)p[k].cols, 0, (int8_t)g[k].type, (int8_t)(copies ? copies[k].type : 0)};
    };
    const auto small = [&](int32_t k) { return fits<16>(p[k].rows, p[k].cols); };
    std::vector<Group> groups;
    int64_t x = 0, s = 0, pieces = 0;
    for (int kind = 0; kind < 4; ++kind) {
        const bool tall = kind & 1, tiny = kind & 2;
        bool open = false;
        for (int32_t k = 0; k < n; ++k) {
            const int64_t rows = p[k].rows, cols = p[k].cols, side = std::min(rows, cols);
            const int64_t values = rows * padded(cols);
            if (rows * cols == 0 || small(k) || (rows > cols) != tall || (side < 8) != tiny) continue;
            if (open && (groups.back().job.count == kGroup || groups.back().x + values > kGroupValues)) open = false;
            if (!open) {
                groups.push_back(Group{});
                groups.back().tall = tall;
                groups.back().tiny = tiny;
                open = true;
            }
            Group& q = groups.back();
            q.pieces += (uint32_t)ceil_div(rows * cols, kPiece);
            Matrix t = describe(k);
            t.x = q.x;
            t.s = q.s;
            t.piece_end = q.pieces;
            q.job.t[q.job.count++] = t;
            q.x += values;
            q.s += side * padded(side);
        }
    }
    for (Group& q : groups) {
        q.splits = choose_splits(ctx, q);
        x = std::max(x, q.x);
        s = std::max(s, (q.splits + 1) * q.s);   // G's splits, then P
        pieces = std::max<int64_t>(pieces, q.pieces);
    }
    double* part = nullptr;
    float *xs = nullptr, *ss = nullptr;
    if (!groups.empty()) {
        part = (double*)gs_malloc(ctx, 8 * pieces, GS_MEM_SCRATCH, tmp);
        xs = (float*)gs_malloc(ctx, 4 * 2 * x, GS_MEM_SCRATCH, tmp);
        ss = (float*)gs_malloc(ctx, 4 * s, GS_MEM_SCRATCH, tmp);
        if (!part || !xs || !ss) return GS_ERR_OOM;
    }
    GsTimerScope ts(ctx, "muon");
    for (int large = 0; large < 2; ++large) {
        Job job{};
        for (int32_t k = 0; k <= n; ++k) {
            if (k < n && p[k].rows * p[k].cols > 0 && small(k) && !fits<4>(p[k].rows, p[k].cols) == (large == 1))
                job.t[job.count++] = describe(k);
            if (job.count == 0 || (k < n && job.count < kGroup)) continue;
            if (large) hipLaunchKernelGGL(k_small<16>, dim3(job.count), dim3(1024), 0, ctx->stream, job, c, norm, o->steps);
            else hipLaunchKernelGGL(k_small<4>, dim3(job.count), dim3(256), 0, ctx->stream, job, c, norm, o->steps);
            job.count = 0;
        }
    }
    for (const Group& q : groups) {
        float *now = xs, *other = xs + x;
        const dim3 grid(q.pieces), block(kThreads);
        hipLaunchKernelGGL(k_momentum, grid, block, 0, ctx->stream, q.job, c, norm, part);
        hipLaunchKernelGGL(k_start, grid, block, 0, ctx->stream, q.job, c, norm, part, now);
        if (q.tall) newton_schulz<true>(ctx, q, o->steps, &now, &other, ss, ss + q.splits * q.s);
        else newton_schulz<false>(ctx, q, o->steps, &now, &other, ss, ss + q.splits * q.s);
        hipLaunchKernelGGL(k_apply, grid, block, 0, ctx->stream, q.job, c, norm, now);
    }
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}
