// group.hip -- positions of an index list grouped by the table row they name:
// a stable sort of (row, position), the positions ascending within a row.
//
// Up to kRankMax positions: tiles sorted by counting, then merged (one or two
// launches, where the passes below take three each; whole table gradients of
// rows of 8 f32 into 32768 take, so and with passes, 15.2 and 32 us for 4000
// positions, 22.4 and 37 for 32768, 35.8 and 38 for 65536, 57.5 and 38 for
// 98304).  More: one to four passes of up to 9 bits of the row, lowest first,
// each a histogram per tile of 4096 positions, a scan of every digit's counts
// over the tiles, and a stable scatter; the first pass reads the indices
// themselves.  6M positions by 16 bits: 95 us, two passes of 10 us (histogram),
// 5 (scan) and 33 (scatter, 96 MB moved; tiles of 8192 took 38).  Positions
// that name no row (masked, padding) have a digit of their own after all
// others in every pass, so that they end up last without a bit of the key.
#include "gs_device.h"
#include "gs_internal.h"
#include "gs_tensor.h"

#include <algorithm>
#include <type_traits>

namespace {

using gst::row_of;

// Tiles of 2048 positions, each sorted by counting: position i of a tile goes
// to the place
//   #{j : key_j < key_i} + #{j < i : key_j = key_i} = #{j < i : key_j < key_i + 1} + #{j > i : key_j < key_i}
// over the tile, one compare and one add per pair.  A block ranks 64 positions
// (one per lane); its 16 wavefronts each count a sixteenth of the tile's keys,
// which are staged in LDS and read four at a time by all lanes from one
// address.
constexpr int kRankThreads = 1024, kRankWaves = kRankThreads / 64;
constexpr int kRankTile = 2048;
template <typename I>
__global__ __launch_bounds__(kRankThreads) void k_group_rank(const I* __restrict__ idx, int n, uint32_t rows,
                                                             int64_t skip, uint32_t* __restrict__ keys,
                                                             uint32_t* __restrict__ pos)
{
    __shared__ uint4 sk4[kRankTile / 4];
    __shared__ uint32_t cnt[kRankWaves][64];
    uint32_t* sk = reinterpret_cast<uint32_t*>(sk4);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int s = (int)(blockIdx.x / (kRankTile / 64)) * kRankTile, m = min(kRankTile, n - s);   // the tile
    for (int j = threadIdx.x; j < kRankTile; j += kRankThreads)
        sk[j] = j < m ? row_of(idx, s + j, rows, skip) : 0xFFFFFFFFu;
    __syncthreads();
    const int i0 = (int)blockIdx.x * 64 - s, i = i0 + lane;
    const uint32_t ki = i < m ? sk[i] : 0u;
    uint32_t c = 0;
    auto count = [&](int qa, int qb, uint32_t thr) {
#pragma unroll 4
        for (int q = qa; q < qb; ++q) {
            const uint4 k = sk4[q];
            c += (k.x < thr ? 1u : 0u) + (k.y < thr ? 1u : 0u) + (k.z < thr ? 1u : 0u) + (k.w < thr ? 1u : 0u);
        }
    };
    const int m4 = (m + 3) / 4, per = (m4 + kRankWaves - 1) / kRankWaves;
    const int q0 = min(m4, wave * per), q1 = min(m4, q0 + per);
    const int b0 = i0 / 4, b1 = b0 + 16;   // the block's own
    count(q0, min(q1, b0), ki + 1u);
    for (int q = max(q0, b0); q < min(q1, b1); ++q) {
        const uint4 k = sk4[q];
        c += (k.x < ki + (4 * q < i ? 1u : 0u) ? 1u : 0u) + (k.y < ki + (4 * q + 1 < i ? 1u : 0u) ? 1u : 0u) +
             (k.z < ki + (4 * q + 2 < i ? 1u : 0u) ? 1u : 0u) + (k.w < ki + (4 * q + 3 < i ? 1u : 0u) ? 1u : 0u);
    }
    count(max(q0, b1), q1, ki);
    cnt[wave][lane] = c;
    __syncthreads();
    if (wave == 0 && i < m) {
        uint32_t r = 0;
        for (int w = 0; w < kRankWaves; ++w) r += cnt[w][lane];
        keys[s + r] = ki;
        pos[s + r] = (uint32_t)(s + i);
    }
}

// Sorted tiles merged: an element's place is its place in its own tile, plus,
// for every tile before, the elements with keys up to its own, and for every
// tile after, those with smaller keys, each found by bisection.  A block takes
// 64 neighbours of a tile (their bisections follow nearly the same path); its
// wavefronts share the other tiles.
constexpr int kMergeWaves = 8;
__global__ __launch_bounds__(64 * kMergeWaves) void k_group_merge(const uint32_t* __restrict__ kin,
                                                                 const uint32_t* __restrict__ pin, int n,
                                                                 uint32_t* __restrict__ keys,
                                                                 uint32_t* __restrict__ pos)
{
    __shared__ uint32_t cnt[kMergeWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int own = (int)(blockIdx.x / (kRankTile / 64)), tiles = (n + kRankTile - 1) / kRankTile;
    const int i = (int)blockIdx.x * 64 + lane;
    const uint32_t ki = i < n ? kin[i] : 0u;
    uint32_t c = 0;
    for (int t = wave; t < tiles; t += kMergeWaves) {
        if (t == own) continue;
        const uint32_t thr = ki + (t < own ? 1u : 0u);   // count the keys < thr
        const uint32_t* k = kin + t * kRankTile;
        const int m = min(kRankTile, n - t * kRankTile);
        // lane l holds the last key of the tile's l-th part: a bisection over
        // the lanes finds the part, one in memory the place in it
        constexpr int kPart = kRankTile / 64;
        const uint32_t last = lane * kPart + kPart <= m ? k[lane * kPart + kPart - 1] : 0xFFFFFFFFu;
        int part = 0;
#pragma unroll
        for (int step = 32; step > 0; step >>= 1)
            if ((uint32_t)__shfl((int)last, part + step - 1, 64) < thr) part += step;
        // part <= 63, and all keys of parts before it are < thr; if the last
        // lane's is too, every key is
        int lo = part * kPart;
#pragma unroll
        for (int step = kPart; step > 0; step >>= 1)
            if (lo + step <= m && k[min(lo + step, m) - 1] < thr) lo += step;
        c += (uint32_t)lo;
    }
    cnt[wave][lane] = c;
    __syncthreads();
    if (wave == 0 && i < n) {
        uint32_t r = (uint32_t)(i - own * kRankTile);
        for (int w = 0; w < kMergeWaves; ++w) r += cnt[w][lane];
        keys[r] = ki;
        pos[r] = pin[i];
    }
}

// ---------------------------------------------------------------------------
// The passes.  A tile is 8 wavefronts of 8 rounds of 64 positions; a
// wavefront's positions are consecutive.  FIRST: the pass reads the indices,
// the others the lists of the pass before.
constexpr int kThreads = 512, kWaves = kThreads / 64, kItems = 8, kTile = kThreads * kItems;
constexpr int kMaxBits = 9;
constexpr int kBins = 1 << kMaxBits;   // digits; bin `1 << bits` (at most kBins) holds what names no row

struct Pass {
    const uint32_t* keys;
    const uint32_t* pos;
    int64_t n, tiles;
    uint32_t rows;
    int64_t skip;
    int shift, bits;
};

template <typename I, bool FIRST>
__device__ __forceinline__ uint32_t key_at(const Pass& a, const I* __restrict__ idx, int64_t i)
{
    if constexpr (FIRST) return row_of(idx, i, a.rows, a.skip);
    else return a.keys[i];
}

__device__ __forceinline__ uint32_t bin_of(const Pass& a, uint32_t key)
{
    return key < a.rows ? (key >> a.shift) & ((1u << a.bits) - 1u) : 1u << a.bits;
}

template <typename I, bool FIRST>
__global__ __launch_bounds__(kThreads) void k_group_hist(const I* __restrict__ idx, Pass a, uint32_t* __restrict__ hist)
{
    // eight copies, taken by the lanes in turn: a row that many positions
    // name does not hold up the counting
    constexpr int kCopies = 8, kStep = kBins + 5;
    __shared__ uint32_t h[kCopies * kStep];
    const int bins = (1 << a.bits) + 1;
    for (int d = threadIdx.x; d < kCopies * kStep; d += kThreads) h[d] = 0u;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kTile + threadIdx.x;
    uint32_t k[kItems];
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        k[r] = key_at<I, FIRST>(a, idx, min(base + r * kThreads, a.n - 1));
    }
#pragma unroll
    for (int r = 0; r < kItems; ++r)
        if (base + r * kThreads < a.n) atomicAdd(&h[(threadIdx.x % kCopies) * kStep + bin_of(a, k[r])], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += kThreads) {
        uint32_t all = 0;
#pragma unroll
        for (int q = 0; q < kCopies; ++q) all += h[q * kStep + d];
        hist[(int64_t)d * a.tiles + blockIdx.x] = all;
    }
}

// exclusive scan of v over the block's threads
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* sh, uint32_t* total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t x = v;
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t y = __shfl_up(x, o, 64);
        if (lane >= o) x += y;
    }
    if (lane == 63) sh[wave] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int w = 0; w < (int)blockDim.x / 64; ++w) {
        if (w < wave) before += sh[w];
        all += sh[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

// one block per digit: its counts become the counts of the tiles before
__global__ __launch_bounds__(256) void k_group_scan(uint32_t* __restrict__ hist, int64_t tiles,
                                                    uint32_t* __restrict__ total)
{
    __shared__ uint32_t sh[4];
    uint32_t* row = hist + (int64_t)blockIdx.x * tiles;
    uint32_t carry = 0;
    for (int64_t t0 = 0; t0 < tiles; t0 += 1024) {
        uint32_t v[4], own = 0, all;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t t = t0 + 4 * threadIdx.x + q;
            v[q] = t < tiles ? row[t] : 0u;
            own += v[q];
        }
        uint32_t at = carry + block_scan(own, sh, &all);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t t = t0 + 4 * threadIdx.x + q;
            if (t < tiles) row[t] = at;
            at += v[q];
        }
        carry += all;
    }
    if (threadIdx.x == 0) total[blockIdx.x] = carry;
}

// Each wavefront ranks its positions among its own, round by round: the lanes
// with one digit are found with a ballot per bit, and a counter per
// (wavefront, digit) in LDS carries the count over the rounds without a
// barrier.  The counters are then scanned over the wavefronts, the tile is put
// in digit order in LDS, and written out so that neighbouring lanes write
// neighbouring places.
template <typename I, bool FIRST>
__global__ __launch_bounds__(kThreads) void k_group_scatter(const I* __restrict__ idx, Pass a,
                                                            const uint32_t* __restrict__ hist,
                                                            const uint32_t* __restrict__ total,
                                                            uint32_t* __restrict__ keys, uint32_t* __restrict__ pos)
{
    __shared__ uint16_t cnt[kWaves][kBins + 1];
    __shared__ uint32_t to[kBins + 1];      // place of the tile's first of each digit, minus its place in the tile
    __shared__ uint16_t local[kBins + 1];   // its place in the tile
    __shared__ uint32_t sh[kWaves];
    __shared__ uint32_t sk[kTile], sp[kTile];
    const int bins = (1 << a.bits) + 1;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int d = lane; d < bins; d += 64) cnt[wave][d] = 0;
    const int64_t first = (int64_t)blockIdx.x * kTile, w0 = first + wave * (64 * kItems);
    uint32_t k[kItems], p[kItems], d[kItems], rank[kItems];
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const int64_t i = min(w0 + 64 * r + lane, a.n - 1);
        k[r] = key_at<I, FIRST>(a, idx, i);
        p[r] = FIRST ? (uint32_t)i : a.pos[i];
    }
    gsd::wave_sync();
    const uint64_t below = (1ull << lane) - 1ull;
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const bool valid = w0 + 64 * r + lane < a.n;
        d[r] = bin_of(a, k[r]);
        uint64_t same = gsd::ballot(valid);
        for (int b = 0; b <= a.bits; ++b) {
            const bool one = (d[r] >> b) & 1u;
            const uint64_t set = gsd::ballot(one);
            same &= one ? set : ~set;
        }
        const uint32_t before = valid ? cnt[wave][d[r]] : 0u;
        rank[r] = before + (uint32_t)__popcll(same & below);
        gsd::wave_sync();   // every lane has read its counter
        if (valid && (same & below) == 0) cnt[wave][d[r]] = (uint16_t)(before + (uint32_t)__popcll(same));
        gsd::wave_sync();
    }
    __syncthreads();
    // per digit: the wavefronts' counts become the counts before them; the
    // digit's place in the tile and in the whole
    uint32_t base = 0, wbase = 0;
    for (int q0 = 0; q0 < bins; q0 += kThreads) {
        uint32_t own = 0, all, tot = 0, wall;
        const int q = q0 + threadIdx.x;
        if (q < bins) {
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t c = cnt[w][q];
                cnt[w][q] = (uint16_t)own;
                own += c;
            }
            tot = total[q];
        }
        const uint32_t at = base + block_scan(own, sh, &all);
        const uint32_t whole = wbase + block_scan(tot, sh, &wall);
        if (q < bins) {
            local[q] = (uint16_t)at;
            to[q] = whole + hist[(int64_t)q * a.tiles + blockIdx.x] - at;
        }
        base += all;
        wbase += wall;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        if (w0 + 64 * r + lane < a.n) {
            const uint32_t at = local[d[r]] + cnt[wave][d[r]] + rank[r];
            sk[at] = k[r];
            sp[at] = p[r];
        }
    }
    __syncthreads();
    const int m = (int)min((int64_t)kTile, a.n - first);
    for (int q = threadIdx.x; q < m; q += kThreads) {
        const uint32_t key = sk[q];
        const uint32_t o = to[bin_of(a, key)] + (uint32_t)q;
        keys[o] = key;
        pos[o] = sp[q];
    }
}

}  // namespace

// positions up to which tiles are counted and merged (the times above)
constexpr int64_t kRankMax = 65536;

gs_status launch_group(gs_ctx* ctx, const void* idx, int idx_type, int64_t n, int64_t rows, int64_t skip,
                       std::vector<GsAlloc>* tmp, GsGroups* out, bool allocate)
{
    const int64_t m = ceil_div(std::max<int64_t>(n, 1), 8) * 8;
    const bool rank = n <= kRankMax, merge = rank && n > kRankTile;
    const int64_t tiles = ceil_div(n, kTile);
    if (allocate) {
        out->keys = (uint32_t*)gs_malloc(ctx, 4 * m, GS_MEM_SCRATCH, tmp);
        out->pos = (uint32_t*)gs_malloc(ctx, 4 * m, GS_MEM_SCRATCH, tmp);
        bool ok = out->keys && out->pos;
        if (!rank || merge) {
            out->keys2 = (uint32_t*)gs_malloc(ctx, 4 * m, GS_MEM_SCRATCH, tmp);
            out->pos2 = (uint32_t*)gs_malloc(ctx, 4 * m, GS_MEM_SCRATCH, tmp);
            ok = ok && out->keys2 && out->pos2;
        }
        if (!rank) {
            out->hist = (uint32_t*)gs_malloc(ctx, 4 * (kBins + 1) * (tiles + 1), GS_MEM_SCRATCH, tmp);
            ok = ok && out->hist;
        }
        return ok ? GS_OK : GS_ERR_OOM;
    }
    if (n == 0) return GS_OK;
    GsTimerScope ts(ctx, "group");
    auto go = [&](auto i) {
        using I = decltype(i);
        if (rank) {
            hipLaunchKernelGGL((k_group_rank<I>), dim3((unsigned)ceil_div(n, 64)), dim3(kRankThreads), 0, ctx->stream,
                               (const I*)idx, (int)n, (uint32_t)rows, skip, out->keys, out->pos);
            if (merge) {
                hipLaunchKernelGGL(k_group_merge, dim3((unsigned)ceil_div(n, 64)), dim3(64 * kMergeWaves), 0,
                                   ctx->stream, out->keys, out->pos, (int)n, out->keys2, out->pos2);
                std::swap(out->keys, out->keys2);
                std::swap(out->pos, out->pos2);
            }
            return;
        }
        const int bits = std::max(1, bits_for(rows));
        const int passes = (bits + kMaxBits - 1) / kMaxBits, step = (bits + passes - 1) / passes;
        uint32_t* const total = out->hist + (kBins + 1) * tiles;
        Pass a{nullptr, nullptr, n, tiles, (uint32_t)rows, skip, 0, 0};
        for (int s = 0; s < bits; s += step) {
            a.shift = s;
            a.bits = std::min(step, bits - s);
            auto pass = [&](auto first) {
                constexpr bool FIRST = decltype(first)::value;
                hipLaunchKernelGGL((k_group_hist<I, FIRST>), dim3((unsigned)tiles), dim3(kThreads), 0, ctx->stream,
                                   (const I*)idx, a, out->hist);
                hipLaunchKernelGGL(k_group_scan, dim3((1u << a.bits) + 1u), dim3(256), 0, ctx->stream, out->hist,
                                   tiles, total);
                hipLaunchKernelGGL((k_group_scatter<I, FIRST>), dim3((unsigned)tiles), dim3(kThreads), 0, ctx->stream,
                                   (const I*)idx, a, out->hist, total, out->keys2, out->pos2);
            };
            if (s == 0) pass(std::true_type{});
            else pass(std::false_type{});
            std::swap(out->keys, out->keys2);
            std::swap(out->pos, out->pos2);
            a.keys = out->keys;
            a.pos = out->pos;
        }
    };
    if (idx_type == GS_I32) go(int32_t{});
    else go(int64_t{});
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}
