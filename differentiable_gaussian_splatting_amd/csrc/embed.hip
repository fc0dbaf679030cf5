// embed.hip -- rows of a table by index, and the table's gradient.
//
//   forward   out[i, c] = scale table[idx[i], c]
//   backward  dtable[v, c] = scale sum over {i : idx[i] = v} of dout[i, c]
//
// Both move memory and compute next to nothing.  Forward, 6M x 48 f32 from
// 65536 rows: 254 us, 4.7 TB/s of indices, table and output; with a table that
// stays in one XCD's L2 (500 rows) 169 us, 6.9 TB/s, the rate of plain stores;
// the 12.6 MB table does not (4 MB a piece), and its reads from the last cache
// bound the call.  16384 x 4096 bf16: 29 us.
//
// The backward groups the positions i by index with a stable sort, so that
// each row's sum runs over its positions in a fixed order and needs no
// atomics: the result does not depend on timing.  6M x 48 f32 (rows 59 apart,
// a quarter of them on one table row): 465 us, of which the sums take 359: a
// row of 192 bytes that starts anywhere touches 2.5 lines of 128 bytes, 2.0 GB
// in all at 5.6 TB/s; the grouping takes 95 and the join 12.  16384 x 4096
// bf16 into 32768 rows of f32: 145 us, of which the sums with the cleared rows
// take 121-131 (671 MB, 5.1-5.5 TB/s).  257 x 45 f32: 9.6 us, one launch.
#include "gs_device.h"
#include "gs_internal.h"
#include "gs_tensor.h"

#include <algorithm>
#include <type_traits>

namespace {

using gst::narrow;
using gst::row_of;
using gst::with_type;

// The rows of out are cut into packs of VEC values (16 bytes of the wider
// type); the last pack of a row whose width is no multiple of VEC starts
// earlier and repeats some of the values before it.  A thread looks up one
// pack, so that a wavefront writes 1 KB of neighbouring packs (two, four and
// eight packs in flight per thread took 261, 266 and 267 us where one takes
// 254, 6M x 48 f32), with stores that do not stay in the L2 (336 us with plain
// ones, which push the table out of it).  Pack k of a block is in row
// (rem + k) / per_row from the block's first row: a product with `magic`
// (floor(2^32 / per_row) + 1, exact for k per_row < 2^32) where
// 1 < per_row < 1024, else a compare (a block then meets at most two rows).
struct FwdShape {
    int64_t n;             // rows of out
    uint32_t rows, cols;
    uint32_t per_row, magic;
    int64_t tstride, ostride;
    float scale;
};

template <typename T, typename O, typename I, int VEC>
__global__ __launch_bounds__(256) void k_embed_fwd(const T* __restrict__ table, const I* __restrict__ idx,
                                                   O* __restrict__ out, FwdShape sh)
{
    const int64_t base = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256;
    const int64_t row0 = base / sh.per_row;
    const uint32_t k = (uint32_t)(base - row0 * sh.per_row) + threadIdx.x;
    const uint32_t r = sh.per_row == 1     ? k
                       : sh.per_row < 1024 ? __umulhi(k, sh.magic)
                                           : (k >= sh.per_row ? 1u : 0u);
    const int64_t row = row0 + r;
    if (row >= sh.n) return;
    const uint32_t col = min((k - r * sh.per_row) * VEC, sh.cols - VEC);
    const uint32_t src = row_of(idx, row, sh.rows, -1);
    gst::Pack<O, VEC> y;
    if (src < sh.rows) {
        const auto x = gst::load<T, VEC>(table + (int64_t)src * sh.tstride + col);
#pragma unroll
        for (int e = 0; e < VEC; ++e) y.v[e] = narrow<O>(sh.scale * (float)x.v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) y.v[e] = (O)0.0f;
    }
    gst::store_once<O, VEC>(out + row * sh.ostride + col, y);
}

// ---------------------------------------------------------------------------
// The backward: (1) the positions sorted by (row, position), group.hip; (2)
// sums over chunks of sorted positions, and zeros in the rows without a
// position; (3) the runs that cross blocks joined.

// the index list, for the sums that sort it themselves
struct Index {
    const void* p;
    int64_t skip;
    int type;
    __device__ __forceinline__ uint32_t row(int64_t i, uint32_t rows) const
    {
        return type == GS_I32 ? row_of((const int32_t*)p, i, rows, skip) : row_of((const int64_t*)p, i, rows, skip);
    }
};

// How (2) and (3) split the sorted positions and the columns.  A team of
// `1 << lg` lanes, each holding VEC neighbouring columns (16 bytes), adds up
// the rows of `chunk` positions; a block's 256 >> lg teams take neighbouring
// chunks.
struct SumShape {
    const uint32_t* keys;   // [n] rows in ascending order, `rows` for what is left out
    const uint32_t* pos;    // [n] positions, ascending within a row
    int64_t n;
    uint32_t rows, cols;
    int lg;
    int chunk;              // a multiple of 8
    int64_t per_block;      // chunk * teams
    uint32_t blocks;        // blocks of positions
    uint32_t slabs;         // column ranges of (1 << lg) VEC columns
    int zero_rows;          // table rows that a wavefront clears where they have no position
    float* head;            // [blocks][cols] sum of the run that reaches a block from before
    float* tail;            // [blocks][cols] sum of the run that starts in a block and goes on after it
};

struct Dest {
    void* p;
    int64_t stride;
    int type, accumulate;
    float scale;
};

// This lane's columns of row v: scale s (+ old), rounded once.  The last lane
// of a row whose width is no multiple of VEC loads and sums some columns of the
// lane before it (cb < c0): it stores them too, the same bits, but does not add
// them to the old values a second time.
template <typename O, int VEC>
__device__ __forceinline__ void put_row(const Dest& d, uint32_t v, uint32_t c0, uint32_t cb, const float* s)
{
    O* o = (O*)d.p + (int64_t)v * d.stride + cb;
    gst::Pack<O, VEC> r;
    if (!d.accumulate) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) r.v[e] = narrow<O>(d.scale * s[e]);
        gst::store<O, VEC>(o, r);
    } else if (cb == c0) {
        r = gst::load<O, VEC>(o);
#pragma unroll
        for (int e = 0; e < VEC; ++e) r.v[e] = narrow<O>((float)r.v[e] + d.scale * s[e]);
        gst::store<O, VEC>(o, r);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (cb + e >= c0) o[e] = narrow<O>((float)o[e] + d.scale * s[e]);
    }
}

// the same columns of a row of f32 partials
template <int VEC>
__device__ __forceinline__ void put_part(float* row, uint32_t c0, uint32_t cb, const float* s)
{
    if (cb == c0) {
        gst::Pack<float, VEC> r;
#pragma unroll
        for (int e = 0; e < VEC; ++e) r.v[e] = s[e];
        gst::store<float, VEC>(row + c0, r);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (cb + e >= c0) row[cb + e] = s[e];
    }
}

// Which of the rows [v0, v0 + zero_rows) have no position, a bit each: every
// lane looks one of them up in the sorted keys.
__device__ __forceinline__ uint64_t unused_rows(const SumShape& sh, int64_t v0)
{
    const int lane = threadIdx.x & 63;
    const int64_t v = v0 + lane;
    bool unused = lane < sh.zero_rows && v < (int64_t)sh.rows;
    if (unused) {
        int64_t lo = 0, hi = sh.n;
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (sh.keys[mid] < (uint32_t)v) lo = mid + 1;
            else hi = mid;
        }
        unused = lo == sh.n || sh.keys[lo] != (uint32_t)v;
    }
    return gsd::ballot(unused);
}

// The same from a short list of indices: the lanes read all of them.
__device__ __forceinline__ uint64_t unnamed_rows(const SumShape& sh, const Index& idx, int64_t v0)
{
    const int lane = threadIdx.x & 63;
    uint64_t named = 0;
    for (int64_t j = lane; j < sh.n; j += 64) {
        const uint32_t r = idx.row(j, sh.rows);
        const int64_t rel = (int64_t)r - v0;
        if (r < sh.rows && rel >= 0 && rel < 64) named |= 1ull << rel;
    }
    for (int o = 1; o < 64; o <<= 1) named |= (uint64_t)__shfl_xor((unsigned long long)named, o, 64);
    const int64_t there = min((int64_t)sh.zero_rows, (int64_t)sh.rows - v0);
    const uint64_t rows = there <= 0 ? 0ull : there >= 64 ? ~0ull : (1ull << there) - 1ull;
    return rows & ~named;
}

// zeros in the rows v0 + r of dtable whose bit r of `left` is set, by one wavefront
__device__ __forceinline__ void clear_rows(const SumShape& sh, const Dest& d, int64_t v0, uint64_t left)
{
    const int lane = threadIdx.x & 63;
    const gst::Pack<uint16_t, 8> zero{};
    const int esize = d.type == GS_F32 ? 4 : 2;
    const int64_t bytes = (int64_t)sh.cols * esize;
    // teams of 1 << zlg lanes, 16 bytes a lane, take the rows in turn
    int zlg = 0;
    while (zlg < 6 && (16ll << zlg) < bytes) ++zlg;
    const int zteam = lane >> zlg, zlane = lane & ((1 << zlg) - 1), zteams = 64 >> zlg;
    for (int r = zteam; r < sh.zero_rows; r += zteams) {
        if (!((left >> r) & 1ull)) continue;
        char* row = (char*)d.p + (v0 + r) * d.stride * esize;
        for (int64_t q = 16 * zlane; q < bytes; q += 16 << zlg) {
            if (q + 16 <= bytes) gst::store_once(reinterpret_cast<uint16_t*>(row + q), zero);
            else
                for (int64_t e = q; e < bytes; e += 2) *reinterpret_cast<uint16_t*>(row + e) = 0;
        }
    }
}

// (2) Bound by the rows' random reads.  A team's lanes hold 16 bytes of a row
// each, so that a row is read in one piece, and chunks of positions instead of
// table rows are shared out, so that a row that many positions name costs no
// more than others (a thread per table row took 645 ms with a quarter of 6M
// positions on one).  Each team walks its chunk in batches, eight rows in
// flight (the loads must not be behind branches: waiting for each in turn took
// 470 us where this takes 359), and adds rows while the table row stays the
// same.  A run inside the chunk is written at once.  A chunk's first run, if
// it began before, is its head, and its last, if it goes on, its tail.  After
// the block's teams are done, the heads that belong to one run are added over
// the teams by doubling steps, and the team in which the run begins adds its
// tail and writes the row, or the block's piece of it (head / tail) if the run
// leaves the block.  Blocks after those of the positions clear the unused
// rows, in the same launch so that their stores run beside the loads.
//
// TINY: up to kTiny positions that one block of 1024 threads holds in one
// batch per team.  The block sorts them itself, by counting as in group.hip, so
// that a small gradient is one launch.
constexpr int kBatch = 8, kTiny = 512;
__device__ __forceinline__ void sort_tiny(const Index& idx, int n, uint32_t rows, uint32_t* keys, uint32_t* pos)
{
    __shared__ uint4 raw4[kTiny / 4];
    __shared__ uint32_t cnt[2][kTiny];
    uint32_t* raw = reinterpret_cast<uint32_t*>(raw4);
    const int t = threadIdx.x, i = t % kTiny, half = t / kTiny, i0 = i & ~63;   // 1024 threads: two per position
    if (half == 0) raw[i] = i < n ? idx.row(i, rows) : 0xFFFFFFFFu;
    __syncthreads();
    const uint32_t ki = raw[i];
    const int n4 = (n + 3) / 4, q0 = half ? (n4 + 1) / 2 : 0, q1 = half ? n4 : (n4 + 1) / 2;
    const int b0 = i0 / 4, b1 = b0 + 16;   // the wavefront's own positions
    uint32_t c = 0;
    auto count = [&](int qa, int qb, uint32_t thr) {
#pragma unroll 4
        for (int q = qa; q < qb; ++q) {
            const uint4 k = raw4[q];
            c += (k.x < thr ? 1u : 0u) + (k.y < thr ? 1u : 0u) + (k.z < thr ? 1u : 0u) + (k.w < thr ? 1u : 0u);
        }
    };
    if (i0 < n) {
        count(q0, min(q1, b0), ki + 1u);
        for (int q = max(q0, b0); q < min(q1, b1); ++q) {
            const uint4 k = raw4[q];
            c += (k.x < ki + (4 * q < i ? 1u : 0u) ? 1u : 0u) + (k.y < ki + (4 * q + 1 < i ? 1u : 0u) ? 1u : 0u) +
                 (k.z < ki + (4 * q + 2 < i ? 1u : 0u) ? 1u : 0u) + (k.w < ki + (4 * q + 3 < i ? 1u : 0u) ? 1u : 0u);
        }
        count(max(q0, b1), q1, ki);
    }
    cnt[half][i] = c;
    __syncthreads();
    if (half == 0 && i < n) {
        const uint32_t r = cnt[0][i] + cnt[1][i];
        keys[r] = ki;
        pos[r] = (uint32_t)i;
    }
    __syncthreads();
}

template <typename T, typename O, int VEC, bool TINY>
__global__ __launch_bounds__(TINY ? 1024 : 256) void k_embed_sum(const T* __restrict__ dout, int64_t dstride,
                                                                SumShape sh, Dest d, Index idx)
{
    constexpr int kT = TINY ? 1024 : 256;
    __shared__ float heads[kT * VEC];
    __shared__ uint8_t on_from[kT];   // per team: its head's run goes on behind what is added so far
    const uint32_t sums = sh.blocks * sh.slabs;
    if (blockIdx.x >= sums) {
        const int64_t v0 = ((int64_t)(blockIdx.x - sums) * (kT / 64) + (threadIdx.x >> 6)) * sh.zero_rows;
        clear_rows(sh, d, v0, TINY ? unnamed_rows(sh, idx, v0) : unused_rows(sh, v0));
        return;
    }
    const uint32_t *keys = sh.keys, *pos = sh.pos;
    if constexpr (TINY) {
        __shared__ uint32_t tk[kTiny], tp[kTiny];
        sort_tiny(idx, (int)sh.n, sh.rows, tk, tp);
        keys = tk;
        pos = tp;
    }
    const uint32_t blk = blockIdx.x / sh.slabs, slab = blockIdx.x - blk * sh.slabs;
    const int lanes = 1 << sh.lg, teams = kT >> sh.lg;
    const int team = threadIdx.x >> sh.lg, lane = threadIdx.x & (lanes - 1);
    const uint32_t c0 = (slab * lanes + lane) * VEC;
    const bool on = c0 < sh.cols;                                  // this lane has columns
    const uint32_t cb = min(c0, sh.cols - VEC);                    // where it loads them (cols >= VEC)
    const int64_t s = (int64_t)blk * sh.per_block + (int64_t)team * sh.chunk;
    const int64_t e = min(sh.n, s + sh.chunk);
    float acc[VEC], head[VEC];
    bool has_head = false, has_tail = false, through = false;   // through: the head is all of the chunk, and goes on
    uint32_t cur = sh.rows;
#pragma unroll
    for (int q = 0; q < VEC; ++q) head[q] = 0.0f;
    if (s < e) {
        // the lists are padded to whole batches
        auto k = gst::load<uint32_t, kBatch>(keys + s);
        auto p = gst::load<uint32_t, kBatch>(pos + s);
        const uint32_t before = s > 0 ? keys[s - 1] : sh.rows, after = e < sh.n ? keys[e] : sh.rows;
        cur = k.v[0];
        const bool from = before == cur;
        bool in_first = true;
#pragma unroll
        for (int q = 0; q < VEC; ++q) acc[q] = 0.0f;
        const T* col = dout + cb;
        for (int64_t j = s; j < e && cur < sh.rows; j += kBatch) {
            // a place past the chunk or without a row reads row 0, and its
            // value is left out below: loads without branches, so that all
            // eight are in flight
            gst::Pack<T, VEC> x[kBatch];
            uint32_t kk[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                kk[b] = j + b < e ? k.v[b] : sh.rows;
                const uint32_t r = kk[b] < sh.rows ? p.v[b] : 0u;
                x[b] = gst::load<T, VEC>(col + (int64_t)r * dstride);
            }
            const int64_t jn = min(j + kBatch, (e - 1) / kBatch * kBatch);   // the last batch again at the end
            k = gst::load<uint32_t, kBatch>(keys + jn);
            p = gst::load<uint32_t, kBatch>(pos + jn);
            if (kk[kBatch - 1] == cur) {   // keys ascend: all of the batch
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
#pragma unroll
                    for (int q = 0; q < VEC; ++q) acc[q] += (float)x[b].v[q];
                }
                continue;
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (kk[b] >= sh.rows) continue;
                if (kk[b] != cur) {   // the run of `cur` ends here
                    if (in_first && from) {
                        has_head = true;
#pragma unroll
                        for (int q = 0; q < VEC; ++q) head[q] = acc[q];
                    } else if (on) {
                        put_row<O, VEC>(d, cur, c0, cb, acc);
                    }
                    in_first = false;
                    cur = kk[b];
#pragma unroll
                    for (int q = 0; q < VEC; ++q) acc[q] = 0.0f;
                }
#pragma unroll
                for (int q = 0; q < VEC; ++q) acc[q] += (float)x[b].v[q];
            }
        }
        if (cur < sh.rows) {
            if (in_first && from) {
                has_head = true;
                through = after == cur;
#pragma unroll
                for (int q = 0; q < VEC; ++q) head[q] = acc[q];
            } else if (after == cur) {
                has_tail = true;
            } else if (on) {
                put_row<O, VEC>(d, cur, c0, cb, acc);
            }
        }
    }
    // heads of one run, added over the teams t .. t + 2 step - 1 while it goes on
    bool goes = through;
    auto publish = [&]() {
#pragma unroll
        for (int q = 0; q < VEC; ++q) heads[threadIdx.x * VEC + q] = head[q];
        if (lane == 0) on_from[team] = goes;
        __syncthreads();
    };
    if (__syncthreads_or(through)) {
        for (int step = 1; step < teams; step <<= 1) {
            publish();
            if (goes && team + step < teams) {
                const float* h = heads + (threadIdx.x + (step << sh.lg)) * VEC;
#pragma unroll
                for (int q = 0; q < VEC; ++q) head[q] += h[q];
                goes = on_from[team + step];
            }
            __syncthreads();
        }
    }
    publish();
    if (!on) return;
    if (team == 0 && has_head) put_part<VEC>(sh.head + (int64_t)blk * sh.cols, c0, cb, head);
    if (has_tail) {
        bool leaves = true;
        if (team + 1 < teams) {
            const float* h = heads + (threadIdx.x + (1 << sh.lg)) * VEC;
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[q] += h[q];
            leaves = on_from[team + 1];
        }
        if (leaves) put_part<VEC>(sh.tail + (int64_t)blk * sh.cols, c0, cb, acc);
        else put_row<O, VEC>(d, cur, c0, cb, acc);
    }
}

// (3) One block per border between blocks of (2) and column range, most of
// which end at once: if a run begins in the block before it and crosses the
// border, its tail and the heads of the blocks after it are added, the teams
// taking every teams-th piece, their sums in order.
template <int VEC>
__global__ __launch_bounds__(256) void k_embed_join(SumShape sh, Dest d)
{
    __shared__ float part[256 * VEC];
    __shared__ uint32_t more[4];
    const uint32_t slab = blockIdx.x % sh.slabs;
    const int64_t b = blockIdx.x / sh.slabs, end = (b + 1) * sh.per_block;
    const uint32_t row = sh.keys[end];   // end < n: only inner borders are launched
    if (row >= sh.rows || sh.keys[end - 1] != row) return;
    if (b > 0 && sh.keys[b * sh.per_block - 1] == row) return;   // it began earlier
    // blocks b + 1 .. b + m hold its heads: block t does if the key at its start is row
    const int64_t blocks = sh.blocks;
    int64_t m = 0;
    for (;;) {
        const int64_t t = b + 1 + m + threadIdx.x;
        const uint64_t yes = gsd::ballot(t < blocks && sh.keys[t * sh.per_block] == row);
        if ((threadIdx.x & 63) == 0) more[threadIdx.x >> 6] = (uint32_t)__popcll(yes);
        __syncthreads();
        const uint32_t got = more[0] + more[1] + more[2] + more[3];
        __syncthreads();
        m += got;
        if (got < 256) break;
    }
    const int lanes = 1 << sh.lg, teams = 256 >> sh.lg;
    const int team = threadIdx.x >> sh.lg, lane = threadIdx.x & (lanes - 1);
    const uint32_t c0 = (slab * lanes + lane) * VEC;
    const bool on = c0 < sh.cols;
    const uint32_t cb = min(c0, sh.cols - VEC);
    float acc[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) acc[q] = 0.0f;
    if (on) {
        // piece 0 is the tail, piece t the head of block b + t; eight in flight
        const float* heads = sh.head + b * sh.cols + cb;
        if (team == 0) {
            const auto x = gst::load<float, VEC>(sh.tail + b * sh.cols + cb);
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[q] = x.v[q];
        }
        int64_t t = team == 0 ? teams : team;
        for (; t + 7 * teams <= m; t += 8 * teams) {
            gst::Pack<float, VEC> x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = gst::load<float, VEC>(heads + (t + u * teams) * sh.cols);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
#pragma unroll
                for (int q = 0; q < VEC; ++q) acc[q] += x[u].v[q];
            }
        }
        for (; t <= m; t += teams) {
            const auto x = gst::load<float, VEC>(heads + t * sh.cols);
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[q] += x.v[q];
        }
    }
#pragma unroll
    for (int q = 0; q < VEC; ++q) part[threadIdx.x * VEC + q] = acc[q];
    __syncthreads();
    if (!on || team != 0) return;
    for (int t = 1; t < teams && t <= m; ++t) {
#pragma unroll
        for (int q = 0; q < VEC; ++q) acc[q] += part[((t << sh.lg) + lane) * VEC + q];
    }
    if (d.type == GS_F32) put_row<float, VEC>(d, row, c0, cb, acc);
    else if (d.type == GS_F16) put_row<gst::f16, VEC>(d, row, c0, cb, acc);
    else put_row<gst::bf16, VEC>(d, row, c0, cb, acc);
}

}  // namespace

gs_status launch_embed_fwd(gs_ctx* ctx, const gs_tensor* table, const void* idx, int idx_type, int64_t n, float scale,
                           const gs_tensor* out)
{
    const int64_t cols = table->cols;
    if (n == 0 || cols == 0) return GS_OK;
    const int most = table->type == GS_F32 || out->type == GS_F32 ? 4 : 8;
    int vec = 1;
    while (2 * vec <= most && 2 * vec <= cols) vec *= 2;
    FwdShape sh{};
    sh.n = n;
    sh.rows = (uint32_t)table->rows;
    sh.cols = (uint32_t)cols;
    sh.per_row = (uint32_t)ceil_div(cols, vec);
    sh.magic = sh.per_row > 1 ? (uint32_t)((1ull << 32) / sh.per_row) + 1u : 0u;
    const int64_t packs = n * sh.per_row, blocks = ceil_div(packs, 256);
    sh.tstride = table->stride;
    sh.ostride = out->stride;
    sh.scale = scale;
    // a launch takes fewer than 2^32 threads in x
    const int64_t gx = std::min<int64_t>(blocks, 1 << 22), gy = ceil_div(blocks, gx);
    if (gy > 65535)
        return gs_fail(ctx, GS_ERR_OVERFLOW, "lookup of %lld x %lld values", (long long)n, (long long)cols);
    GsTimerScope ts(ctx, "embed_fwd");
    auto go = [&](auto t, auto o, auto i, auto v) {
        using T = decltype(t);
        using O = decltype(o);
        using I = decltype(i);
        hipLaunchKernelGGL((k_embed_fwd<T, O, I, decltype(v)::value>), dim3((unsigned)gx, (unsigned)gy),
                           dim3(256), 0, ctx->stream, (const T*)table->data, (const I*)idx, (O*)out->data, sh);
    };
    with_type(table->type, [&](auto t) {
        with_type(out->type, [&](auto o) {
            auto sized = [&](auto v) {
                if (idx_type == GS_I32) go(t, o, int32_t{}, v);
                else go(t, o, int64_t{}, v);
            };
            if (vec == 1) sized(std::integral_constant<int, 1>{});
            else if (vec == 2) sized(std::integral_constant<int, 2>{});
            else if (vec == 4) sized(std::integral_constant<int, 4>{});
            else if constexpr (sizeof(t) == 2 && sizeof(o) == 2) sized(std::integral_constant<int, 8>{});
        });
    });
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

gs_status launch_embed_bwd(gs_ctx* ctx, const void* idx, int idx_type, int64_t n, const gs_tensor* dout, float scale,
                           int64_t padding, int accumulate, const gs_tensor* dtable, std::vector<GsAlloc>* tmp)
{
    const int64_t rows = dtable->rows, cols = dtable->cols;
    if (rows == 0 || cols == 0 || (n == 0 && accumulate)) return GS_OK;
    // the split: columns per lane (16 bytes of dout, or fewer in narrow
    // rows), lanes per team, positions per team
    int vec = 1, lg = 0;
    auto split = [&](int most) {
        for (vec = 1; 2 * vec <= most && 2 * vec <= cols;) vec *= 2;
        for (lg = 0; lg < 6 && (int64_t)vec << lg < cols;) ++lg;
    };
    // few positions: one launch (a block of 1024 threads, whose registers hold
    // packs of four values) instead of two, up to about 320 positions (x 4 f32:
    // 200 positions 8.9 us against 10.4, 300 10.3 against 10.5, 384 11.3 against
    // 10.6), or instead of three, where the other form needs a join, up to what
    // the block holds (x 48: 200 positions 8.7 against 14.4, 512 13.4 against 14.7)
    split(4);
    const bool joined = n > (int64_t)kBatch * (256 >> lg);
    // a launch has fewer than 2^32 threads: with rows of 2^28 columns or more
    // the smaller blocks take the column ranges
    const bool tiny = n > 0 && n <= std::min<int64_t>(joined ? kTiny : 320, kBatch * (1024 >> lg)) && cols < 1 << 28;
    if (!tiny) split(dout->type == GS_F32 ? 4 : 8);
    const int64_t slabs = ceil_div(cols, (int64_t)vec << lg);
    // sixteen wavefronts for each compute unit, in chunks of 8 to 256 positions
    const int64_t want = (n * slabs << lg) / (64 * 16 * (int64_t)ctx->num_cu);
    SumShape sh{};
    sh.n = n;
    sh.rows = (uint32_t)rows;
    sh.cols = (uint32_t)cols;
    sh.lg = lg;
    sh.chunk = (int)std::min<int64_t>(256, std::max<int64_t>(kBatch, want / kBatch * kBatch));
    sh.per_block = (int64_t)sh.chunk * (256 >> lg);
    if (tiny) {
        sh.chunk = kBatch;
        sh.per_block = (int64_t)kBatch * (1024 >> lg);
    }
    const int64_t blocks = ceil_div(n, sh.per_block);
    // a wavefront clears about 64 KB
    const int64_t row_bytes = cols * (dtable->type == GS_F32 ? 4 : 2);
    sh.zero_rows = (int)std::min<int64_t>(64, std::max<int64_t>(1, 65536 / row_bytes));
    const int64_t clear = accumulate ? 0 : ceil_div(rows, (tiny ? 16 : 4) * (int64_t)sh.zero_rows);
    if (blocks * slabs + clear > 0xFFFFFF)   // 2^32 threads
        return gs_fail(ctx, GS_ERR_OVERFLOW, "table gradient of %lld rows of %lld values", (long long)rows,
                       (long long)cols);
    sh.blocks = (uint32_t)blocks;
    sh.slabs = (uint32_t)slabs;

    GsGroups groups;
    gs_status st = tiny ? GS_OK : launch_group(ctx, idx, idx_type, n, rows, padding, tmp, &groups, true);
    if (st != GS_OK) return st;
    if (blocks > 1) {
        sh.head = (float*)gs_malloc(ctx, 4 * blocks * cols, GS_MEM_SCRATCH, tmp);
        sh.tail = (float*)gs_malloc(ctx, 4 * blocks * cols, GS_MEM_SCRATCH, tmp);
        if (!sh.head || !sh.tail) return GS_ERR_OOM;
    }
    if (!tiny) st = launch_group(ctx, idx, idx_type, n, rows, padding, tmp, &groups, false);
    if (st != GS_OK) return st;
    sh.keys = groups.keys;
    sh.pos = groups.pos;
    const Dest d{dtable->data, dtable->stride, dtable->type, accumulate, scale};
    GsTimerScope ts(ctx, "embed_sum");
    auto sum = [&](auto t, auto v) {
        using T = decltype(t);
        constexpr int VEC = decltype(v)::value;
        auto launch = [&](auto o, auto small) {
            using O = decltype(o);
            constexpr bool TINY = decltype(small)::value;
            hipLaunchKernelGGL((k_embed_sum<T, O, VEC, TINY>), dim3((unsigned)(blocks * slabs + clear)),
                               dim3(TINY ? 1024 : 256), 0, ctx->stream, (const T*)dout->data, dout->stride, sh, d,
                               Index{idx, padding, idx_type});
        };
        with_type(dtable->type, [&](auto o) {
            if (!tiny) launch(o, std::false_type{});
            else if constexpr (VEC <= 4) launch(o, std::true_type{});
        });
        if (blocks > 1)
            hipLaunchKernelGGL((k_embed_join<VEC>), dim3((unsigned)((blocks - 1) * slabs)), dim3(256), 0, ctx->stream,
                               sh, d);
    };
    with_type(dout->type, [&](auto t) {
        if (vec == 1) sum(t, std::integral_constant<int, 1>{});
        else if (vec == 2) sum(t, std::integral_constant<int, 2>{});
        else if (vec == 4) sum(t, std::integral_constant<int, 4>{});
        else if constexpr (sizeof(t) == 2) sum(t, std::integral_constant<int, 8>{});
    });
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}
