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
//
// The products bound it: 3 matrices of 4096 x 4096 12.9 to 13.6 ms, all but 0.4
// of it products at 295 to 360 TFLOP/s (three f16 products each; G and P by half
// their tiles); 24 of 2048 x 515 1.6 to 1.75 ms, where a fifth to a third of the
// tiles is padding and each splits its f32 values again at every step of k.  A
// few matrices of 64 x 48 take one launch and 24 us, fifteen products that wait
// for each other.
#include <algorithm>
#include <cmath>

#include "gs_internal.h"
#include "gs_tensor.h"
#include "mm.h"
#include "muon_plan.h"

namespace {

using namespace gsm;

typedef gst::Pack<float, 4> Four;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr double kEps = 1e-7;
constexpr float kScaleX = 32768.0f, kScaleP = 16384.0f;   // of X and G, and of P

constexpr int kThreads = 256;
constexpr int kPiece = 4096;      // values of a block of the elementwise kernels
constexpr int kGroup = 48;        // matrices of a launch (kernel arguments within 4 KB)

// A matrix of a group.  Its X, G and P start at x, s and s in the group's
// workspaces, with zeros around them up to whole tiles of the group (unit):
// the products need no edges, and the zeros stay zeros.
struct Matrix {
    float *p, *m;
    const void* g;
    void* copy;
    int64_t gld;
    int64_t x, s;
    int32_t rows, cols;
    uint32_t piece_end;           // pieces of the matrices up to this one
    uint32_t start_end;           // of their padded X
    int8_t gtype, ctype;
};
struct Job {
    Matrix t[kGroup];
    int32_t count;
    int32_t unit;                 // to whose multiples the sides in the workspaces are rounded up
};
struct MuonConst {
    float mu, lr, keep;           // keep = 1 - lr weight_decay
    int32_t nesterov;
};

struct Shape {
    int64_t x, s;
    int32_t rows, cols;           // padded
    int32_t side, length;         // the shorter and the longer side up to a whole step of k: beyond are zeros
    uint32_t tile_end;            // tiles of the matrices up to this one
};
struct MmJob {
    Shape t[kGroup];
    int32_t count;
};
static_assert(sizeof(Job) <= 3904 && sizeof(MmJob) <= 3904, "kernel arguments");

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

// The calling thread's values of a piece, four neighbours at a time:
// f(flat index, values, row, column of the first).
template <typename F>
__device__ __forceinline__ void each_four(int64_t n, int32_t cols, uint32_t piece, F&& f)
{
    const int64_t first = (int64_t)piece * kPiece, end = min(n, first + kPiece);
    const int32_t down = kThreads * 4 / cols, along = kThreads * 4 % cols;
    int64_t i = first + threadIdx.x * 4, r = i / cols;
    int32_t c = (int32_t)(i - r * cols);
#pragma unroll 2
    for (; i < end; i += kThreads * 4) {
        f(i, (int)min((int64_t)4, end - i), r, c);
        r += down;
        c += along;
        if (c >= cols) {
            c -= cols;
            ++r;
        }
    }
}

// four neighbours from (r, c) on of a matrix whose rows are ld apart
template <typename S>
__device__ __forceinline__ f32x4 four_of(const S* p, int64_t ld, int32_t cols, int64_t i, int valid, int64_t r, int32_t c)
{
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (ld == cols && valid == 4) {
        const gst::Pack<S, 4> x = gst::load<S, 4>(p + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (float)x.v[j];
        return v;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j < valid) v[j] = (float)p[r * ld + c];
        if (++c == cols) {
            c = 0;
            ++r;
        }
    }
    return v;
}

__device__ __forceinline__ f32x4 four_gradients(const Matrix& t, int64_t i, int valid, int64_t r, int32_t c)
{
    f32x4 v;
    with_type_device(t.gtype, [&](auto s) { v = four_of((const decltype(s)*)t.g, t.gld, t.cols, i, valid, r, c); });
    return v;
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

// 1 / (|u| + eps) from the sum of squares, as two factors: |u| may be anything up
// to 2^21 times the largest float, and its inverse less than a normal float.
__device__ __forceinline__ float2 inverse_norm(double squares)
{
    const double d = sqrt(squares) + kEps;
    const double down = d > 0x1p100 ? 0x1p-64 : 1.0;
    return make_float2((float)(1.0 / (d * down)), (float)down);
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
    each_four((int64_t)t.rows * t.cols, t.cols, blockIdx.x - before, [&](int64_t i, int valid, int64_t r, int32_t c) {
        const f32x4 g = f * four_gradients(t, i, valid, r, c);
        const f32x4 m = o.mu * four_of(t.m, t.cols, t.cols, i, valid, r, c) + g;
        const f32x4 u = o.nesterov ? g + o.mu * m : m;
        if (valid == 4) {
            gst::store<float, 4>(t.m + i, __builtin_bit_cast(Four, m));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < valid) t.m[i + j] = m[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += j < valid ? (double)u[j] * u[j] : 0.0;
    });
    sum = block_sum<4>(sum, sums);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// X = u / (|u| + eps), zeros around it; a block per piece of padded X
__global__ __launch_bounds__(kThreads) void k_start(const Job job, const MuonConst o, const float* __restrict__ norm,
                                                    const double* __restrict__ part, float* __restrict__ x)
{
    __shared__ double sums[4];
    if (norm && !isfinite(norm[0])) return;
    const float f = norm ? norm[1] : 1.0f;
    uint32_t before;
    const int k = matrix_of(job, blockIdx.x, [](const Matrix& q) { return q.start_end; }, before);
    const Matrix& t = job.t[k];
    double sum = 0.0;
    for (uint32_t b = (k ? job.t[k - 1].piece_end : 0u) + threadIdx.x; b < t.piece_end; b += kThreads) sum += part[b];
    const float2 inv = inverse_norm(block_sum<4>(sum, sums));
    const int32_t ld = (int32_t)padded(t.cols, job.unit);
    each_four(padded(t.rows, job.unit) * ld, ld, blockIdx.x - before, [&](int64_t i, int, int64_t r, int32_t c) {
        const int valid = r < t.rows ? min(4, t.cols - c) : 0;   // ld is a multiple of 4: the four share a row
        f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f};
        if (valid > 0) {
            const int64_t at = r * t.cols + c;
            u = four_of(t.m, t.cols, t.cols, at, valid, r, c);
            if (o.nesterov) {
                f32x4 g;
                with_type_device(t.gtype, [&](auto s) {
                    typedef decltype(s) S;
                    g = four_of((const S*)t.g + r * t.gld, t.cols, t.cols, c, valid, 0, c);
                });
                u = f * g + o.mu * u;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = j < valid ? u[j] * inv.x * inv.y : 0.0f;
        }
        *reinterpret_cast<f32x4*>(x + t.x + i) = u;
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
    const int32_t ld = (int32_t)padded(t.cols, job.unit);
    each_four((int64_t)t.rows * t.cols, t.cols, blockIdx.x - before, [&](int64_t i, int valid, int64_t r, int32_t c) {
        const f32x4 p = four_of(t.p, t.cols, t.cols, i, valid, r, c) * o.keep -
                        rate * four_of(x + t.x, ld, t.cols, i, valid, r, c);
        if (valid == 4) {
            gst::store<float, 4>(t.p + i, __builtin_bit_cast(Four, p));
            if (!t.copy) return;
            with_type_device(t.ctype, [&](auto s) {
                typedef decltype(s) S;
                gst::Pack<S, 4> v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v.v[j] = gst::narrow<S>(p[j]);
                gst::store<S, 4>((S*)t.copy + i, v);
            });
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < valid) write_parameter(t, i + j, p[j]);
        }
    });
}

// One tile of a matrix's product: G (kGram), P from G (kPoly) or the next X.
// G and P are symmetric: their tiles on and below the diagonal are computed and
// those below it written to both places.  Sides are the padded ones.
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
    const int64_t side = TALL ? t.cols : t.rows;
    const int64_t m = KIND == kNext ? t.rows : side, n = KIND == kNext ? t.cols : side;
    int64_t i, j;
    if constexpr (KIND == kNext) {
        tile_at(b - before, m / T::BM, n / T::BN, i, j);
    } else {
        static_assert(T::BM == T::BN, "square tiles");
        const int q = (int)(b - before);
        int r = (int)((sqrtf(8.0f * (float)q + 1.0f) - 1.0f) * 0.5f);
        while (r * (r + 1) / 2 > q) --r;
        while ((r + 1) * (r + 2) / 2 <= q) ++r;
        i = r;
        j = q - r * (r + 1) / 2;
    }
    const float* src = from + (KIND == kPoly ? t.s : t.x);
    const Operand x = {src, KIND == kPoly ? side : t.cols, 0, kScaleX, 0};
    Operand a = x, bo = x;
    if constexpr (KIND == kNext) (TALL ? bo : a) = Operand{poly + t.s, side, 0, kScaleP, 0};
    a.rows = m;
    bo.rows = n;
    f32x4 acc[T::NI][T::MI];
#pragma unroll
    for (int q = 0; q < T::NI; ++q)
#pragma unroll
        for (int r = 0; r < T::MI; ++r) acc[q][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    int64_t k0 = 0, k1 = KIND == kGram ? t.length : t.side;
    if constexpr (KIND == kGram) {
        const int64_t each = (t.length / T::BK + splits - 1) / splits * T::BK;
        k0 = min((int64_t)t.length, split * each);
        k1 = min((int64_t)t.length, k0 + each);
    }
    mm_tile<float, 2, ACOL, BCOL, T, true>(a, bo, i * T::BM, j * T::BN, k0, k1, lds, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row0 = i * T::BM + (wave % T::WM) * T::MI * 16 + (lane & 15);
    const int64_t col0 = j * T::BN + (wave / T::WM) * T::NI * 16 + (lane >> 4) * 4;
    const float down = 1.0f / kScaleX / (KIND == kNext ? kScaleP : kScaleX);
    float* dst = to + (KIND == kNext ? t.x : t.s) + (KIND == kGram ? split * split_size : 0);
#pragma unroll
    for (int r = 0; r < T::MI; ++r) {
#pragma unroll
        for (int q = 0; q < T::NI; ++q) {
            const int64_t row = row0 + r * 16, col = col0 + q * 16, at = row * n + col;
            f32x4 y = acc[q][r] * down;
            if constexpr (KIND != kGram) {
                const f32x4 old = *reinterpret_cast<const f32x4*>(src + at);
                y = KIND == kPoly ? kC * y + kB * old : y + kA * old;
            }
            *reinterpret_cast<f32x4*>(dst + at) = y;
            if (KIND != kNext && i != j) {
#pragma unroll
                for (int w = 0; w < 4; ++w) dst[(col + w) * n + row] = y[w];
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
typedef Tile<64, 64, 64, 2, 2, 1> Small;

static_assert(Large::BM == kNewtonCosts[0].b && Medium::BM == kNewtonCosts[1].b && Small::BM == kNewtonCosts[2].b, "tiles");

// the matrices whose products share launches, and the floats of their X and G
struct Group {
    Job job;
    int64_t x, s;
    uint32_t pieces, starts;
    bool tall;                    // more rows than columns
    int splits;                   // of G's products
};

template <int KIND, bool TALL, typename T>
void launch_tiles(gs_ctx* ctx, const Group& q, const float* from, float* to, const float* poly)
{
    const int splits = KIND == kGram ? q.splits : 1, unit = q.job.unit;
    MmJob mm{};
    uint32_t tiles = 0;
    for (int32_t k = 0; k < q.job.count; ++k) {
        const Matrix& t = q.job.t[k];
        tiles += (uint32_t)tiles_of<KIND>(t, unit, T::BM);
        mm.t[mm.count++] = Shape{t.x, t.s, (int32_t)padded(t.rows, unit), (int32_t)padded(t.cols, unit),
                               (int32_t)padded(std::min(t.rows, t.cols), T::BK), (int32_t)padded(std::max(t.rows, t.cols), T::BK),
                               tiles};
    }
    hipLaunchKernelGGL((k_newton<KIND, TALL, T>), dim3(tiles * splits), dim3(T::NT), 0, ctx->stream, mm, from, to, poly,
                       splits, q.s);
    if (splits > 1)
        hipLaunchKernelGGL(k_sum_splits, dim3((uint32_t)std::min<int64_t>(ceil_div(q.s, 4 * kThreads), 2048)),
                           dim3(kThreads), 0, ctx->stream, to, q.s, splits);
}

template <int KIND, bool TALL>
void launch_newton(gs_ctx* ctx, const Group& q, const float* from, float* to, const float* poly)
{
    double us;
    const int tile = choose_tile<KIND>(ctx->num_cu, q.job, q.job.unit, KIND == kGram ? q.splits : 1, &us);
    if (tile == 0) launch_tiles<KIND, TALL, Large>(ctx, q, from, to, poly);
    else if (tile == 1) launch_tiles<KIND, TALL, Medium>(ctx, q, from, to, poly);
    else launch_tiles<KIND, TALL, Small>(ctx, q, from, to, poly);
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
    const int64_t s = padded(std::min(rows, cols), 32), l = padded(std::max(rows, cols), 32);
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
    const int S = (int)padded(s, 32), L = (int)padded(l, 32), ldx = L + 8, ldg = S + 8;
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
    const float2 inv = inverse_norm(block_sum<W>(sum, lds.sums));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) x[i][j] = x[i][j] * inv.x * inv.y;
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
                      (int32_t)p[k].rows, (int32_t)p[k].cols, 0, 0, (int8_t)g[k].type, (int8_t)(copies ? copies[k].type : 0)};
    };
    const auto small = [&](int32_t k) { return fits<16>(p[k].rows, p[k].cols); };
    std::vector<Group> groups;
    int64_t x = 0, s = 0, pieces = 0;
    for (int tall = 0; tall < 2; ++tall) {
        bool open = false;
        int64_t held = 0;
        for (int32_t k = 0; k < n; ++k) {
            const int64_t rows = p[k].rows, cols = p[k].cols;
            if (rows * cols == 0 || small(k) || (rows > cols) != (tall == 1)) continue;
            const int64_t values = padded(rows, 64) * padded(cols, 64);
            if (open && (groups.back().job.count == kGroup || held + values > kGroupValues)) open = false;
            if (!open) {
                groups.push_back(Group{});
                groups.back().tall = tall == 1;
                open = true;
                held = 0;
            }
            held += values;
            Job& job = groups.back().job;
            job.t[job.count++] = describe(k);
        }
    }
    for (Group& q : groups) {
        choose_sizes(ctx->num_cu, q.job, &q.job.unit, &q.splits);
        for (int32_t k = 0; k < q.job.count; ++k) {
            Matrix& t = q.job.t[k];
            const int64_t rows = padded(t.rows, q.job.unit), cols = padded(t.cols, q.job.unit), side = std::min(rows, cols);
            t.x = q.x;
            t.s = q.s;
            q.x += rows * cols;
            q.s += side * side;
            t.piece_end = q.pieces += (uint32_t)ceil_div((int64_t)t.rows * t.cols, kPiece);
            t.start_end = q.starts += (uint32_t)ceil_div(rows * cols, kPiece);
        }
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
        hipLaunchKernelGGL(k_start, dim3(q.starts), block, 0, ctx->stream, q.job, c, norm, part, now);
        if (q.tall) newton_schulz<true>(ctx, q, o->steps, &now, &other, ss, ss + q.splits * q.s);
        else newton_schulz<false>(ctx, q, o->steps, &now, &other, ss, ss + q.splits * q.s);
        hipLaunchKernelGGL(k_apply, grid, block, 0, ctx->stream, q.job, c, norm, now);
    }
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}
