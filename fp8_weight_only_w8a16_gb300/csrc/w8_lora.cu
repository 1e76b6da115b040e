// w8_lora.cu -- low-rank adapters of many requests beside a shared projection:
// out[t] = y[t] + s_a B_a (A_a x[t]), rows in the order of their adapters.
//
// Two launches.  The first makes v = A x in fp32: a CTA takes 16 positions of
// one adapter and a range of k, its warps taking 32-column blocks in turn; the
// ranges' partial sums go to the workspace, [range][position][rank].  The
// second adds them in order and multiplies by B: a CTA takes 16 positions of
// one adapter and a run of columns.  Both products are on
// tensor-core steps (mma.sync m16n8k16), far below their rate: the operator is
// bound by its bytes (x, the adapters, y twice), and with few rows by its two
// launches.  Where adapters have rows enough, tiles of 128 positions go through
// both products on tcgen05.
// 54 rows of 30 adapters of rank 32, 16384 to 6144 columns (45 MB): 16 us, two
// launches of a few dependent loads each.  3700 rows of 5 adapters of rank 64, 2048
// to 16384 columns (270 MB): 66 us, 13 of them the first product, 4.1 TB/s.
//
// Operands go from global memory to registers with 16-byte loads: lane (g, t)
// takes 8 consecutive columns of the summed axis, 8t .. 8t+7 of a 32-column
// block, of both operands, which fills two steps whose k slots are these
// columns in an order that is the same on both sides.
#include <limits.h>

#include "w8_grouped_internal.h"
#include "w8_tcgen.cuh"

namespace w8 {

__device__ int g_lora_status;

namespace {

__device__ __forceinline__ void note_timeout() { atomicOr(&g_lora_status, 1); }

constexpr int kLoWarps = 8;
constexpr int kLoThreads = kLoWarps * 32;
constexpr int kShrinkRows = 16;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Tile `want` of those that `rows` positions make, counted through the
// adapters; a whole warp asks.  An adapter begins at the largest offset so far
// (offsets that decrease name no position twice).
struct Tile {
    int adapter, from, count; // adapter -1: there are `count` tiles in all
};
__device__ __forceinline__ Tile find_tile(const w8_lora &a, int want, int rows, int lane)
{
    int at = 0, begin = min(max(__ldg(a.offsets), 0), a.n_rows);
    for (int g0 = 0; g0 < a.n_adapters; g0 += 32) {
        int end = begin;
        if (g0 + lane < a.n_adapters)
            end = max(begin, min(__ldg(a.offsets + g0 + lane + 1), a.n_rows));
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, end, d);
            end = lane >= d ? max(end, o) : end;
        }
        int from = __shfl_up_sync(0xffffffffu, end, 1);
        from = lane ? from : begin;
        const int tiles = (end - from + rows - 1) / rows;
        int inc = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            inc += lane >= d ? o : 0;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, at + inc > want);
        if (here) {
            const int src = __ffs(int(here)) - 1;
            const int k = (want - at - __shfl_sync(0xffffffffu, inc - tiles, src)) * rows;
            end = __shfl_sync(0xffffffffu, end, src);
            from = __shfl_sync(0xffffffffu, from, src) + k;
            return {g0 + src, from, min(end - from, rows)};
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
        begin = __shfl_sync(0xffffffffu, end, 31);
    }
    return {-1, 0, at};
}

// 8 bf16 at columns col .. col+7 of a row of `cols`; zeros past them.
__device__ __forceinline__ uint4 load8(const uint16_t *row, int col, int cols)
{
    if (col + 8 <= cols)
        return __ldg(reinterpret_cast<const uint4 *>(row + col));
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = col + e < cols ? __ldg(row + col + e) : 0u;
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

__device__ __forceinline__ int rank_of(const w8_lora &a, int adapter)
{
    return a.ranks ? min(max(__ldg(a.ranks + adapter), 0), a.rank) : a.rank;
}

// Values from one row to the next in shared memory, 64 bytes more than a multiple
// of 128: eight lanes that read 16 bytes each of two rows then meet no bank twice.
constexpr int row_pitch(int values) { return values % 64 == 32 ? values : values + 32; }

// v of 16 positions over one range of k; kTiles: 16-row tiles of the rank.
template <int kTiles>
__global__ void __launch_bounds__(kLoThreads) shrink_kernel(const __grid_constant__ w8_lora a, float *v, int splits)
{
    extern __shared__ float s_part[]; // [warp][kTiles][2][4][32]
    __shared__ Tile s_tile;
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (warp == 0) {
        const Tile f = find_tile(a, int(blockIdx.x), kShrinkRows, lane);
        if (lane == 0)
            s_tile = f;
    }
    __syncthreads();
    const Tile tile = s_tile;
    if (tile.adapter < 0)
        return;
    const int rank = rank_of(a, tile.adapter);
    const int kb = (a.k + 31) / 32;
    const int b0 = int(int64_t(blockIdx.y) * kb / splits), b1 = int(int64_t(blockIdx.y + 1) * kb / splits);
    const uint16_t *x[2];
    bool xs[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        int row = -1;
        if (8 * j + g < tile.count)
            row = __ldg(a.order + tile.from + 8 * j + g);
        xs[j] = row >= 0 && row < a.n_tok;
        x[j] = a.x + (xs[j] ? row : 0) * a.ldx;
    }
    const uint16_t *w = a.a + tile.adapter * a.ld_a;
    const bool two = tile.count > 8;
    float acc[kTiles][2][4] = {};
#pragma unroll 2
    for (int b = b0 + warp; b < b1; b += kLoWarps) {
        const int col = b * 32 + 8 * t;
        uint4 xv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            xv[j] = xs[j] ? load8(x[j], col, a.k) : make_uint4(0, 0, 0, 0);
        uint4 lo[kTiles], hi[kTiles];
#pragma unroll
        for (int r = 0; r < kTiles; ++r) {
            const int r0 = 16 * r + g, r1 = r0 + 8;
            lo[r] = r0 < rank ? load8(w + r0 * a.ld_a_row, col, a.k) : make_uint4(0, 0, 0, 0);
            hi[r] = r1 < rank ? load8(w + r1 * a.ld_a_row, col, a.k) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < kTiles; ++r) {
            mma16816(acc[r][0], lo[r].x, hi[r].x, lo[r].y, hi[r].y, xv[0].x, xv[0].y);
            mma16816(acc[r][0], lo[r].z, hi[r].z, lo[r].w, hi[r].w, xv[0].z, xv[0].w);
            if (two) {
                mma16816(acc[r][1], lo[r].x, hi[r].x, lo[r].y, hi[r].y, xv[1].x, xv[1].y);
                mma16816(acc[r][1], lo[r].z, hi[r].z, lo[r].w, hi[r].w, xv[1].z, xv[1].w);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kTiles; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s_part[(((warp * kTiles + r) * 2 + j) * 4 + e) * 32 + lane] = acc[r][j][e];
    __syncthreads();
    // accumulator e of lane (g, t): rank row 16 r + g + 8 (e >> 1), position 8 j + 2 t + (e & 1)
    constexpr int kItems = kTiles * 256;
    float *out = v + int64_t(blockIdx.y) * a.n_rows * (16 * kTiles);
    for (int it = threadIdx.x; it < kItems; it += kLoThreads) {
        const int ln = it & 31, e = it >> 5 & 3, j = it >> 7 & 1, r = it >> 8;
        const int pos = 8 * j + 2 * (ln & 3) + (e & 1);
        if (pos >= tile.count)
            continue;
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < kLoWarps; ++q)
            sum += s_part[q * kItems + it];
        out[int64_t(tile.from + pos) * (16 * kTiles) + 16 * r + (ln >> 2) + 8 * (e >> 1)] = sum;
    }
}

// out of 16 positions over `cols` columns; kTiles as above.
template <int kTiles, bool kVec>
__global__ void __launch_bounds__(kLoThreads)
    expand_kernel(const __grid_constant__ w8_lora a, const float *v, int splits, int cols)
{
    constexpr int kBlocks = (kTiles + 1) / 2;      // 32-column blocks of the rank
    constexpr int kPitch = row_pitch(kBlocks * 32);
    constexpr int kPos = 16;
    __shared__ __align__(16) uint16_t s_v[2][kPos * kPitch]; // v as the sum of two bf16
    __shared__ int s_row[kPos];
    __shared__ Tile s_tile;
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (warp == 0) {
        const Tile f = find_tile(a, int(blockIdx.x), kPos, lane);
        if (lane == 0)
            s_tile = f;
    }
    __syncthreads();
    const Tile tile = s_tile;
    if (tile.adapter < 0)
        return;
    const int rank = rank_of(a, tile.adapter);
    const float scale = a.scales ? __ldg(a.scales + tile.adapter) : 1.0f;
    const uint16_t *w = a.b + tile.adapter * a.ld_b;
    const int end = min(int(blockIdx.y + 1) * cols, a.n);
    // 32 columns a warp at a time: step column c of tile j is column
    // 8 (c / 2) + 2 j + c % 2, so that lane (g, t) gets columns 8t .. 8t+7 of
    // its rows' sums
    uint4 bw[kBlocks][4];
    auto load_b = [&](int c0) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = c0 + 8 * (g >> 1) + 2 * j + (g & 1), r0 = 32 * b + 8 * t;
                bw[b][j] = n < a.n && r0 < rank ? load8(w + n * a.ld_b_row, r0, rank) : make_uint4(0, 0, 0, 0);
            }
    };
    const int first = int(blockIdx.y) * cols + 32 * warp;
    if (first < end)
        load_b(first); // on its way while v is joined
    for (int it = threadIdx.x; it < kPos * kBlocks * 32; it += kLoThreads) {
        const int pos = it / (kBlocks * 32), r = it % (kBlocks * 32);
        float sum = 0.0f;
        if (pos < tile.count && r < rank) {
            const float *from = v + int64_t(tile.from + pos) * (16 * kTiles) + r;
            const int64_t step = int64_t(a.n_rows) * (16 * kTiles);
            for (int q = 0; q < splits; ++q)
                sum += __ldcg(from + q * step);
        }
        const uint16_t hi = to_bf16(sum);
        const float h = __uint_as_float(uint32_t(hi) << 16);
        s_v[0][pos * kPitch + r] = hi;
        s_v[1][pos * kPitch + r] = isfinite(h) ? to_bf16(sum - h) : uint16_t(0);
    }
    if (threadIdx.x < kPos) {
        int row = -1;
        if (int(threadIdx.x) < tile.count)
            row = __ldg(a.order + tile.from + threadIdx.x);
        s_row[threadIdx.x] = row < a.n_tok ? row : -1;
    }
    __syncthreads();
    const int row[2] = {s_row[g], s_row[g + 8]};
    for (int c0 = first; c0 < end; c0 += 32 * kLoWarps) {
        const int col = c0 + 8 * t;
        const bool whole = kVec && col + 8 <= a.n;
        uint4 old[2];
        if (whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (row[h] >= 0)
                    old[h] = *reinterpret_cast<const uint4 *>(a.y + row[h] * a.ldy + col);
        }
        float acc[4][4] = {};
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const int r0 = 32 * b + 8 * t;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint16_t *s = s_v[p] + g * kPitch + r0;
                const uint4 lo = *reinterpret_cast<const uint4 *>(s), hi = *reinterpret_cast<const uint4 *>(s + 8 * kPitch);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma16816(acc[j], lo.x, hi.x, lo.y, hi.y, bw[b][j].x, bw[b][j].y);
                    mma16816(acc[j], lo.z, hi.z, lo.w, hi.w, bw[b][j].z, bw[b][j].w);
                }
            }
        }
        if (c0 + 32 * kLoWarps < end)
            load_b(c0 + 32 * kLoWarps);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (row[h] < 0)
                continue;
            uint16_t *out = a.out + row[h] * a.ld_out + col;
            if (whole) {
                const uint32_t o[4] = {old[h].x, old[h].y, old[h].z, old[h].w};
                uint32_t r[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float v0 = fmaf(scale, acc[j][2 * h], __uint_as_float(o[j] << 16));
                    const float v1 = fmaf(scale, acc[j][2 * h + 1], __uint_as_float(o[j] & 0xFFFF0000u));
                    r[j] = to_bf16(v0) | uint32_t(to_bf16(v1)) << 16;
                }
                *reinterpret_cast<uint4 *>(out) = make_uint4(r[0], r[1], r[2], r[3]);
            } else {
                const uint16_t *y = a.y + row[h] * a.ldy + col;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (col + e < a.n)
                        out[e] = to_bf16(fmaf(scale, acc[e / 2][2 * h + (e & 1)], __uint_as_float(uint32_t(y[e]) << 16)));
            }
        }
    }
}

// 16 bytes global -> shared, `bytes` of them read and the others zero.
__device__ __forceinline__ void copy_part(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The same for tiles that are mostly full, on tcgen05: 128 positions over a run of
// columns, 128 at a time.  (With mma.sync the fragments of v and B went through
// registers once a warp: 98 us for 3700 rows of 16384 columns at rank 64, 36 of
// them the bytes of y and out.)
//   D [128 x 128] = V [128 x 2 R] [B | B]^T,  R = 64 or 128: the rank, padded,
// V the two bf16 parts of v beside each other.  The steps of all tiles (128 columns
// of one each) lie in a line, of which every CTA takes an even share: a run of
// columns of a tile, or parts of a few tiles (with a run of one tile a CTA, 124 of
// the SMs had work for 31 tiles).  Thirteen warps, which meet only at their barriers:
// 0-7 join v, add y and store (32 positions by 64 columns each, from tensor memory,
// the sums of the next columns being made meanwhile), 8 copies B (tensor map) and
// issues the steps, 9-12 copy y.  The results go out through y's place in shared
// memory, a row's 128 bytes by eight lanes.  A step takes 1.75 us of all SMs, 5.7
// TB/s of y and out; sixteen warps that store, more stages of B and no tensor-core
// steps at all changed that by 2 % at most.
constexpr int kTcPos = 128, kTcCols = 128;
constexpr int kTcOut = 8, kTcIssue = 8, kTcCopy = 9, kTcCopyWarps = 4;
constexpr int kTcLoraThreads = (kTcCopy + kTcCopyWarps) * 32;
constexpr int kTcPitch = kTcCols * 2 + 16; // bytes of a row of y: 8 rows then meet no bank twice
template <int kRank> struct LoraTc {
    static constexpr int kChunks = kRank / 64;             // 64 values of the rank
    static constexpr int kChunk = 128 * 128;               // bytes of them, of v or B
    static constexpr int kV = 2 * kChunks * kChunk, kB = kChunks * kChunk, kY = kTcPos * kTcPitch;
    static constexpr int kStB = 2, kStY = kRank == 64 ? 3 : 2;
    static constexpr int kSmem = 1024 + kV + kStB * kB + kStY * kY;
    static_assert(kSmem <= 220 * 1024, "shared memory");
};
// A warp's wait.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, tcg::bar_wait(bar, parity));
}
// The row that a position names, -1 for none.
__device__ __forceinline__ int row_at(const w8_lora &a, const Tile &tile, int pos)
{
    const int row = pos < tile.count ? __ldg(a.order + tile.from + pos) : -1;
    return row < a.n_tok ? row : -1;
}
// Ranges of k of a tile's first product: the SMs shared among the tiles, each range at
// least 1024 columns at rank 64 and 2048 at 128, since the second product's CTAs all
// join them (of 256 columns at least: 74 us instead of 66 for 3700 rows of 2048, rank 64).
template <int kRank> __device__ __forceinline__ int tc_splits(int tiles, int k, int sms)
{
    const int want = tiles > 0 ? sms / tiles : 1, most = (k + 63) / 64 / (kRank / 4);
    const int s = want < most ? want : most;
    return s < 1 ? 1 : s < 8 ? s : 8;
}
// Where range q's sums of a tile's position lie in the workspace: with one range in the
// order of the positions, with several by tiles.
__device__ __forceinline__ int64_t sum_row(const Tile &tile, int want, int splits, int q, int pos)
{
    return splits == 1 ? int64_t(tile.from) + pos : (int64_t(want) * splits + q) * kTcPos + pos;
}

// v = A x of the same tiles on tcgen05, each item a tile by a range of k, 64 columns a
// stage: D [128 x R] = X [128 x 64 ..] A^T.  Fourteen warps: 0-3 bring the sums out,
// 4 issues the steps, 5 copies A (tensor map), 6-13 copy the rows of x that the
// positions name into the K-major, 128-byte-swizzled layout (16 bytes a lane, four rows
// a thread and stage).
constexpr int kSxIssue = 4, kSxA = 5, kSxCopy = 6, kSxCopyWarps = 8;
constexpr int kSxThreads = (kSxCopy + kSxCopyWarps) * 32;
template <int kRank> struct ShrinkTc {
    static constexpr int kX = kTcPos * 128, kA = kRank * 128, kStages = kRank == 64 ? 8 : 6;
    static constexpr int kSmem = 1024 + kStages * (kX + kA);
    static_assert(kSmem <= 220 * 1024, "shared memory");
};
template <int kRank>
__global__ void __launch_bounds__(kSxThreads, 1)
    shrink_tc_kernel(const __grid_constant__ w8_lora a, const __grid_constant__ CUtensorMap map_a, float *v, int rank16, int sms)
{
    using namespace tcg;
    using L = ShrinkTc<kRank>;
    constexpr int kStages = L::kStages;
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ __align__(8) uint64_t full_a[kStages], full_x[kStages], used[kStages], sums[2], sums_read[2];
    __shared__ uint32_t s_tmem;
    uint8_t *const s_x = s_dyn + ((1024u - (smem_addr(s_dyn) & 1023u)) & 1023u);
    uint8_t *const s_a = s_x + kStages * L::kX;
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(&full_a[i], 1);
            bar_init(&full_x[i], 32 * kSxCopyWarps);
            bar_init(&used[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sums[i], 1);
            bar_init(&sums_read[i], 4);
        }
        bar_init_fence();
    }
    if (warp == kSxIssue)
        tmem_alloc(&s_tmem, 2 * kRank);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    pdl_launch_dependents();
    pdl_wait();
    bool ok = true;
    const int tiles = find_tile(a, INT_MAX, kTcPos, lane).count, splits = tc_splits<kRank>(tiles, a.k, sms);
    const int chunks = (a.k + 63) / 64, items = tiles * splits;
    uint32_t n = 0; // stages so far
    int c0 = 0, c1 = 0;
    auto range = [&](int id) { // of k, in runs of 64 columns
        const int q = id % splits;
        c0 = int(int64_t(q) * chunks / splits);
        c1 = int(int64_t(q + 1) * chunks / splits);
    };
    if (warp == kSxIssue) {
        constexpr uint32_t idesc = inst_desc(128, kRank, false, false);
        const uint64_t dx = desc128_k(smem_addr(s_x), 1024), da = desc128_k(smem_addr(s_a), 1024);
        uint32_t item = 0;
        for (int id = blockIdx.x; id < items && ok; id += gridDim.x, ++item) {
            range(id);
            const uint32_t part = item & 1u;
            if (item >= 2)
                ok = warp_wait(&sums_read[part], (item / 2 - 1) & 1u);
            for (int c = c0; c < c1 && ok; ++c, ++n) {
                const uint32_t slot = n % kStages, parity = n / kStages & 1u;
                ok = warp_wait(&full_a[slot], parity);
                ok = ok && warp_wait(&full_x[slot], parity);
                if (!ok)
                    break;
                fence_async_shared(); // (x that threads have copied, for the tensor cores)
                fence_after();
                if (elect_one()) {
                    const uint64_t x = dx + uint64_t((slot * L::kX) >> 4), b = da + uint64_t((slot * L::kA) >> 4);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mma_ss(tmem + part * kRank, x + uint64_t((q * 32) >> 4), b + uint64_t((q * 32) >> 4), idesc,
                               uint32_t((c - c0) | q));
                    commit(&used[slot]);
                    if (c + 1 == c1)
                        commit(&sums[part]);
                }
                __syncwarp();
            }
        }
        // every arrival is here before the CTA leaves
        for (uint32_t s = n > kStages ? n - kStages : 0; s < n; ++s)
            ok = warp_wait(&used[s % kStages], s / kStages & 1u) && ok;
    } else if (warp == kSxA) {
        for (int id = blockIdx.x; id < items && ok; id += gridDim.x) {
            range(id);
            const Tile tile = find_tile(a, id / splits, kTcPos, lane);
            for (int c = c0; c < c1; ++c, ++n) {
                const uint32_t slot = n % kStages;
                if (n >= kStages)
                    ok = warp_wait(&used[slot], (n / kStages - 1) & 1u);
                if (!ok)
                    break;
                if (elect_one()) {
                    bar_expect(&full_a[slot], L::kA);
                    copy_box(smem_addr(s_a) + slot * L::kA, &map_a, 64 * c, 0, tile.adapter, &full_a[slot], policy_normal());
                }
                __syncwarp();
            }
        }
        for (uint32_t s = n > kStages ? n - kStages : 0; s < n; ++s) // the copies have landed
            ok = warp_wait(&full_a[s % kStages], s / kStages & 1u) && ok;
    } else if (warp >= kSxCopy) {
        constexpr int kRows = kTcPos / (4 * kSxCopyWarps);
        const int r0 = (threadIdx.x - 32 * kSxCopy) / 8, c8 = 8 * int(threadIdx.x % 8);
        const uint32_t to0 = smem_addr(s_x) + uint32_t(r0 * 128 + ((c8 / 8 ^ (r0 & 7)) << 4));
        for (int id = blockIdx.x; id < items && ok; id += gridDim.x) {
            range(id);
            const Tile tile = find_tile(a, id / splits, kTcPos, lane);
            int row[kRows]; // rows of none keep what the slot held: their sums go nowhere
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                row[i] = row_at(a, tile, r0 + 4 * kSxCopyWarps * i);
            for (int c = c0; c < c1; ++c, ++n) {
                const uint32_t slot = n % kStages;
                if (n >= kStages)
                    ok = warp_wait(&used[slot], (n / kStages - 1) & 1u);
                if (!ok)
                    break;
                const int col = 64 * c + c8, bytes = min(max(2 * (a.k - col), 0), 16);
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (row[i] >= 0)
                        copy_part(to0 + slot * L::kX + uint32_t(i * 4 * kSxCopyWarps * 128), bytes ? a.x + row[i] * a.ldx + col : a.x,
                                  bytes);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&full_x[slot])) : "memory");
            }
        }
        copy16_wait();
    } else {
        uint32_t item = 0;
        for (int id = blockIdx.x; id < items && ok; id += gridDim.x, ++item) {
            const Tile tile = find_tile(a, id / splits, kTcPos, lane);
            const uint32_t part = item & 1u;
            const int pos = 32 * warp + lane;
            ok = warp_wait(&sums[part], item / 2 & 1u);
            if (!ok)
                break;
            fence_after();
            float *const to = v + sum_row(tile, id / splits, splits, id % splits, pos) * rank16;
            for (int r = 0; r < rank16; r += 32) {
                float d[32];
                ld32x32(d, tmem + (uint32_t(32 * warp) << 16) + part * kRank + uint32_t(r));
                wait_ld();
                if (pos < tile.count)
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        if (r + e < rank16)
                            *reinterpret_cast<float4 *>(to + r + e) = make_float4(d[e], d[e + 1], d[e + 2], d[e + 3]);
            }
            fence_before();
            __syncwarp();
            if (lane == 0)
                bar_arrive(&sums_read[part]);
        }
    }
    if (!ok && lane == 0)
        note_timeout();
    fence_before();
    __syncthreads();
    if (warp == kSxIssue) {
        fence_after();
        tmem_free(tmem, 2 * kRank);
    }
}

template <int kRank>
__global__ void __launch_bounds__(kTcLoraThreads, 1)
    expand_tc_kernel(const __grid_constant__ w8_lora a, const __grid_constant__ CUtensorMap map_b, const float *v, int rank16, int sms,
                     int ranges)
{
    using namespace tcg;
    using L = LoraTc<kRank>;
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ __align__(8) uint64_t full_b[L::kStB], free_b[L::kStB], full_y[L::kStY], free_y[L::kStY], sums[2], sums_read[2],
        full_v;
    __shared__ uint32_t s_tmem;
    uint8_t *const s_v = s_dyn + ((1024u - (smem_addr(s_dyn) & 1023u)) & 1023u);
    uint8_t *const s_b = s_v + L::kV, *const s_y = s_b + L::kStB * L::kB;
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kStB; ++i) {
            bar_init(&full_b[i], 1);
            bar_init(&free_b[i], 1);
        }
        for (int i = 0; i < L::kStY; ++i) {
            bar_init(&full_y[i], 32 * kTcCopyWarps);
            bar_init(&free_y[i], kTcOut);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sums[i], 1);
            bar_init(&sums_read[i], kTcOut);
        }
        bar_init(&full_v, kTcOut);
        bar_init_fence();
    }
    if (warp == kTcIssue)
        tmem_alloc(&s_tmem, 2 * kTcCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    pdl_launch_dependents();
    pdl_wait();
    bool ok = true;
    // This CTA's share of the line; every warp looks for its tiles itself.
    const int all = (a.n + kTcCols - 1) / kTcCols;
    const int tiles = find_tile(a, INT_MAX, kTcPos, lane).count;
    const int splits = ranges ? ranges : tc_splits<kRank>(tiles, a.k, sms); // ranges: of shrink_kernel
    const int64_t line = int64_t(tiles) * all;
    int64_t at = line * blockIdx.x / gridDim.x;
    const int64_t until = line * (blockIdx.x + 1) / gridDim.x;
    uint32_t base = 0; // steps of the parts before
    int steps = 0, begin = 0, want = 0;
    // The next part's tile (adapter -1: there is none), its steps and first column.
    auto next = [&] {
        at += steps;
        base += uint32_t(steps);
        if (at >= until)
            return Tile{-1, 0, 0};
        want = int(at / all);
        const int step0 = int(at - int64_t(want) * all);
        steps = int(until - at < all - step0 ? until - at : all - step0);
        begin = step0 * kTcCols;
        return find_tile(a, want, kTcPos, lane);
    };
    if (warp == kTcIssue) {
        constexpr uint32_t idesc = inst_desc(128, kTcCols, false, false);
        const uint64_t dv = desc128_k(smem_addr(s_v), 1024), db = desc128_k(smem_addr(s_b), 1024);
        uint32_t copied = 0, issued = 0, parts = 0;
        for (Tile tile = next(); tile.adapter >= 0 && ok; tile = next(), ++parts) {
            const int rank = rank_of(a, tile.adapter), sixteens = max(1, (rank + 15) / 16);
            const uint32_t end = base + uint32_t(steps);
            auto copy = [&] { // into the slot of the step kStB before, once that is done
                const uint32_t slot = copied % L::kStB;
                if (copied >= L::kStB)
                    ok = ok && warp_wait(&free_b[slot], (copied / L::kStB - 1) & 1u);
                if (!ok)
                    return;
                if (elect_one()) {
                    bar_expect(&full_b[slot], L::kB);
#pragma unroll
                    for (int c = 0; c < L::kChunks; ++c)
                        copy_box(smem_addr(s_b) + slot * L::kB + uint32_t(c * L::kChunk), &map_b, 64 * c,
                                 begin + int(copied - base) * kTcCols, tile.adapter, &full_b[slot], policy_normal());
                }
                __syncwarp();
                ++copied;
            };
            for (int s = 0; s < L::kStB && s < steps; ++s)
                copy();
            ok = ok && warp_wait(&full_v, parts & 1u);
            for (; issued < end && ok; ++issued) {
                const uint32_t slot = issued % L::kStB, part = issued & 1u;
                ok = warp_wait(&full_b[slot], issued / L::kStB & 1u);
                if (issued >= 2)
                    ok = ok && warp_wait(&sums_read[part], (issued / 2 - 1) & 1u);
                if (!ok)
                    break;
                // Steps stop at the adapter's rank; what its rows of B hold past it in
                // the last step is made zero here (past a.rank the copies have done so).
                if (rank < a.rank && rank < 16 * sixteens) {
                    uint8_t *const b = s_b + slot * L::kB + (sixteens - 1) / 4 * L::kChunk;
                    const int eight0 = (sixteens - 1) % 4 * 2, keep = rank - 16 * (sixteens - 1);
                    for (int i = lane; i < 2 * kTcCols; i += 32) { // (row, half of the step)
                        const int row = i >> 1, left = keep - 8 * (i & 1);
                        uint4 *const at16 = reinterpret_cast<uint4 *>(b + row * 128 + (((eight0 + (i & 1)) ^ (row & 7)) << 4));
                        const uint4 old = *at16;
                        auto kept = [&](uint32_t w, int e) {
                            return left > e + 1 ? w : left > e ? w & 0xFFFFu : 0u;
                        };
                        *at16 = make_uint4(kept(old.x, 0), kept(old.y, 2), kept(old.z, 4), kept(old.w, 6));
                    }
                    fence_async_shared();
                    __syncwarp();
                }
                fence_after();
                const uint64_t b = db + uint64_t((slot * L::kB) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int k = 0; k < kRank / 16; ++k)
                            if (k < sixteens)
                                mma_ss(tmem + part * kTcCols, dv + uint64_t(((p * L::kChunks + k / 4) * L::kChunk + (k % 4) * 32) >> 4),
                                       b + uint64_t(((k / 4) * L::kChunk + (k % 4) * 32) >> 4), idesc, uint32_t(p | k));
                    commit(&free_b[slot]);
                    commit(&sums[part]);
                }
                __syncwarp();
                if (copied < end)
                    copy();
            }
        }
        // every copy has landed and every arrival is here before the CTA leaves
        for (uint32_t s = issued > L::kStB ? issued - L::kStB : 0; s < issued; ++s)
            ok = bar_wait(&free_b[s % L::kStB], s / L::kStB & 1u) && ok;
        for (uint32_t s = copied > L::kStB ? copied - L::kStB : 0; s < copied; ++s)
            ok = bar_wait(&full_b[s % L::kStB], s / L::kStB & 1u) && ok;
        ok = __all_sync(0xffffffffu, ok);
    } else if (warp >= kTcCopy) {
        // ---- y: 16 lanes a row's 256 bytes ---------------------------------------------------
        constexpr int kRows = kTcPos / (2 * kTcCopyWarps);
        const int i0 = (threadIdx.x - 32 * kTcCopy) / 16, c8 = 8 * int(threadIdx.x % 16);
        for (Tile tile = next(); tile.adapter >= 0 && ok; tile = next()) {
            int row[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                row[i] = row_at(a, tile, i0 + 2 * kTcCopyWarps * i);
            for (int s = 0; s < steps; ++s) {
                const uint32_t n = base + uint32_t(s), st = n % L::kStY;
                if (n >= L::kStY)
                    ok = warp_wait(&free_y[st], (n / L::kStY - 1) & 1u);
                if (!ok)
                    break;
                const int col = begin + s * kTcCols + c8, bytes = min(max(2 * (a.n - col), 0), 16);
                const uint32_t to = smem_addr(s_y) + st * L::kY + uint32_t(i0 * kTcPitch + c8 * 2);
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (row[i] >= 0)
                        copy_part(to + uint32_t(i * 2 * kTcCopyWarps * kTcPitch), bytes ? a.y + row[i] * a.ldy + col : a.y, bytes);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&full_y[st])) : "memory");
            }
        }
        copy16_wait();
    } else {
        // ---- y + s B v: 32 positions by 64 columns --------------------------------------------
        const int quarter = warp & 3, half = warp >> 2;
        for (Tile tile = next(); tile.adapter >= 0 && ok; tile = next()) {
            const float scale = a.scales ? __ldg(a.scales + tile.adapter) : 1.0f;
            const int rank = rank_of(a, tile.adapter);
            int row[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                row[i] = row_at(a, tile, 32 * quarter + 4 * i + lane / 8);
            // v's two parts, K-major with the 128-byte swizzle: the steps of the part before,
            // whose sums this warp has seen, are through with it
            constexpr int kItems = 4;
            for (int it0 = threadIdx.x; it0 < kTcPos * (kRank / 8); it0 += kItems * 32 * kTcOut) {
                float sum[kItems][8] = {};
#pragma unroll 2
                for (int q = 0; q < splits; ++q)
#pragma unroll
                    for (int i = 0; i < kItems; ++i) {
                        const int it = it0 + i * 32 * kTcOut, pos = it / (kRank / 8), r = 8 * (it % (kRank / 8));
                        if (pos < tile.count && r < rank16) {
                            const float4 *from =
                                reinterpret_cast<const float4 *>(
                                    v + (ranges ? int64_t(q) * a.n_rows + tile.from + pos : sum_row(tile, want, splits, q, pos)) * rank16 + r);
                            const float4 x = __ldcg(from), y = __ldcg(from + 1);
                            const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                sum[i][e] += f[e];
                        }
                    }
#pragma unroll
                for (int i = 0; i < kItems; ++i) {
                    const int it = it0 + i * 32 * kTcOut, pos = it / (kRank / 8), r = 8 * (it % (kRank / 8));
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // (zeros past the rank: 0 x an infinity of x)
                        const float v0 = r + 2 * e < rank ? sum[i][2 * e] : 0.0f, v1 = r + 2 * e + 1 < rank ? sum[i][2 * e + 1] : 0.0f;
                        hi[e] = pack_bf16(v0, v1);
                        const float h0 = __uint_as_float(hi[e] << 16), h1 = __uint_as_float(hi[e] & 0xFFFF0000u);
                        lo[e] = pack_bf16(isfinite(h0) ? v0 - h0 : 0.0f, isfinite(h1) ? v1 - h1 : 0.0f);
                    }
                    uint8_t *to = s_v + (r / 64) * L::kChunk + pos * 128 + (((r % 64) / 8 ^ (pos & 7)) << 4);
                    *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(to + L::kChunks * L::kChunk) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0)
                bar_arrive(&full_v);
            for (int s = 0; s < steps; ++s) {
                const uint32_t n = base + uint32_t(s), st = n % L::kStY;
                const int c0 = begin + s * kTcCols + 64 * half;
                ok = warp_wait(&full_y[st], n / L::kStY & 1u);
                ok = ok && warp_wait(&sums[n & 1], n / 2 & 1u);
                if (!ok)
                    break;
                fence_after();
                uint8_t *const rows = s_y + st * L::kY + 32 * quarter * kTcPitch + 128 * half;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float d[32];
                    ld32x32(d, tmem + (uint32_t(32 * quarter) << 16) + (n & 1) * kTcCols + uint32_t(64 * half + 32 * c));
                    wait_ld();
                    if (c == 1) { // the sums are read
                        fence_before();
                        __syncwarp();
                        if (lane == 0)
                            bar_arrive(&sums_read[n & 1]);
                    }
                    uint4 *mine = reinterpret_cast<uint4 *>(rows + lane * kTcPitch + 64 * c);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 old = mine[q];
                        const uint32_t o[4] = {old.x, old.y, old.z, old.w};
                        uint32_t r[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            r[e] = pack_bf16(fmaf(scale, d[8 * q + 2 * e], __uint_as_float(o[e] << 16)),
                                             fmaf(scale, d[8 * q + 2 * e + 1], __uint_as_float(o[e] & 0xFFFF0000u)));
                        mine[q] = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                }
                __syncwarp();
                const int col = c0 + 8 * (lane % 8);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint8_t *from = rows + (4 * i + lane / 8) * kTcPitch + 16 * (lane % 8);
                    if (row[i] < 0 || col >= a.n)
                        continue;
                    uint16_t *out = a.out + row[i] * a.ld_out + col;
                    if (col + 8 <= a.n) {
                        *reinterpret_cast<uint4 *>(out) = *reinterpret_cast<const uint4 *>(from);
                    } else {
                        for (int e = 0; col + e < a.n; ++e)
                            out[e] = reinterpret_cast<const uint16_t *>(from)[e];
                    }
                }
                __syncwarp();
                if (lane == 0)
                    bar_arrive(&free_y[st]);
            }
        }
    }
    if (!ok && lane == 0)
        note_timeout();
    fence_before();
    __syncthreads();
    if (warp == kTcIssue) {
        fence_after();
        tmem_free(tmem, 2 * kTcCols);
    }
}

// Tiles that n_rows positions of n_adapters adapters can make at most.
int most_tiles(int n_rows, int n_adapters, int rows)
{
    return n_rows / rows + (n_adapters < n_rows ? n_adapters : n_rows);
}

constexpr int shrink_smem(int tiles) { return kLoWarps * tiles * 256 * int(sizeof(float)); }
static_assert(shrink_smem(4) <= 48 * 1024, "no raised limit below eight tiles");

// Every kernel's limit, at the first call on a device.
cudaError_t raise_all()
{
    static std::atomic<uint64_t> raised{0};
    return raise_smem(raised, {{reinterpret_cast<const void *>(&shrink_kernel<8>), shrink_smem(8)},
                               {reinterpret_cast<const void *>(&shrink_tc_kernel<64>), ShrinkTc<64>::kSmem},
                               {reinterpret_cast<const void *>(&shrink_tc_kernel<128>), ShrinkTc<128>::kSmem},
                               {reinterpret_cast<const void *>(&expand_tc_kernel<64>), LoraTc<64>::kSmem},
                               {reinterpret_cast<const void *>(&expand_tc_kernel<128>), LoraTc<128>::kSmem}});
}

int rank_tiles(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

template <int kTiles>
cudaError_t shrink(const w8_lora &a, float *v, int splits, cudaStream_t s)
{
    return launch_dependent(shrink_kernel<kTiles>,
                            dim3(unsigned(most_tiles(a.n_rows, a.n_adapters, kShrinkRows)), unsigned(splits)), kLoThreads,
                            size_t(shrink_smem(kTiles)), s, a, v, splits);
}

template <int kRank>
cudaError_t shrink_tc(const w8_lora &a, float *v, int rank16, int sms, cudaStream_t s)
{
    using L = ShrinkTc<kRank>;
    CUtensorMap map;
    const uint64_t sizes[3] = {uint64_t(a.k), uint64_t(a.rank), uint64_t(a.n_adapters)};
    const uint64_t strides[2] = {uint64_t(a.ld_a_row) * 2, uint64_t(a.n_adapters > 1 ? a.ld_a : a.rank * a.ld_a_row) * 2};
    const uint32_t box[3] = {64, kRank, 1};
    if (!encode_bf16_map(&map, a.a, 3, sizes, strides, box))
        return cudaErrorInvalidValue;
    const int tiles = most_tiles(a.n_rows, a.n_adapters, kTcPos), ctas = int64_t(tiles) * 8 < sms ? tiles * 8 : sms;
    return launch_dependent(shrink_tc_kernel<kRank>, dim3(unsigned(ctas)), kSxThreads, size_t(L::kSmem), s, a, map, v, rank16, sms);
}

template <int kRank>
cudaError_t expand_tc(const w8_lora &a, const float *v, int rank16, int sms, int ranges, cudaStream_t s)
{
    using L = LoraTc<kRank>;
    CUtensorMap map;
    const uint64_t sizes[3] = {uint64_t(a.rank), uint64_t(a.n), uint64_t(a.n_adapters)};
    const uint64_t strides[2] = {uint64_t(a.ld_b_row) * 2, uint64_t(a.n_adapters > 1 ? a.ld_b : a.n * a.ld_b_row) * 2};
    const uint32_t box[3] = {64, kTcCols, 1};
    if (!encode_bf16_map(&map, a.b, 3, sizes, strides, box))
        return cudaErrorInvalidValue;
    const int tiles = most_tiles(a.n_rows, a.n_adapters, kTcPos), steps = (a.n + kTcCols - 1) / kTcCols;
    const int ctas = int64_t(tiles) * steps < sms ? tiles * steps : sms;
    return launch_dependent(expand_tc_kernel<kRank>, dim3(unsigned(ctas)), kTcLoraThreads, size_t(L::kSmem), s, a, map, v, rank16, sms,
                            ranges);
}

template <int kTiles>
cudaError_t lora(const w8_lora &a, float *v, int sms, cudaStream_t s)
{
    const int splits = lora_splits(a.n_rows, a.k, a.n_adapters, sms);
    auto vec = [](const uint16_t *p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; };
    const bool fast = vec(a.y, a.ldy) && vec(a.out, a.ld_out);
    // Tiles of 128 positions where adapters have rows enough.  The host knows the mean
    // only; us with tiles of 128 / 16, rows over adapters (hit, if fewer):
    //                    rank 16    rank 64    rank 32    rank 128
    //                    2048 to 16384 columns 16384-6144 6144-2624
    //   512 over 8       19 / 17    24 / 31    29 / 20    27 / 37
    //   1280 over 40     48 / 40    57 / 69    51 / 48    41 / 77
    //   2560 over 40     60 / 63    67 / 107   61 / 92    53 / 129
    //   2048 over 64 (3) 41 / 50    44 / 88    48 / 84    41 / 73
    constexpr bool kWide = kTiles > 2;
    if (fast && a.n_rows >= (kWide ? 256 : 1024) && a.n_rows >= (kWide ? 32 : 64) * int64_t(a.n_adapters)) {
        constexpr int kRank = kTiles <= 4 ? 64 : 128;
        // The first product by tiles of 16 reads A once for each of them, which for a
        // small A costs less than the ranges' join.  4099 rows of 5 adapters, tiles of 16 /
        // of 128, us, by rank x k (16, 32, 64 or 128 of rank) of
        //   32768   rank 16 of 2048 to 16384                62.3 / 65.5
        //   65536   rank 64 of 1024 to 16384                64.4 / 65.2
        //   131072  rank 64 of 2048 to 16384                69.6 / 70.4
        //           rank 32 of 4096 to 6144                 43.7 / 44.3
        //           rank 16 of 8192 to 6144                 56.7 / 49.2
        //           rank 128 of 1024 to 6144                56.7 / 44.7
        //   262144  rank 64 of 4096 to 6144                 50.2 / 47.5
        //           rank 32 of 8192 to 6144                 60.3 / 51.6
        //           rank 128 of 2048 to 6144                74.1 / 49.6
        const bool small = int64_t(16 * kTiles) * a.k < 131072;
        const cudaError_t e = small ? shrink<kTiles>(a, v, splits, s) : shrink_tc<kRank>(a, v, 16 * kTiles, sms, s);
        return e != cudaSuccess ? e : expand_tc<kRank>(a, v, 16 * kTiles, sms, small ? splits : 0, s);
    }
    const cudaError_t e = shrink<kTiles>(a, v, splits, s);
    if (e != cudaSuccess)
        return e;
    const int tiles = most_tiles(a.n_rows, a.n_adapters, 16);
    constexpr int kStep = 32 * kLoWarps;
    int blocks = (a.n + kStep - 1) / kStep;
    const int per = expand_steps(tiles, blocks, sms);
    blocks = (blocks + per - 1) / per;
    const dim3 grid{unsigned(tiles), unsigned(blocks)};
    return fast ? launch_dependent(expand_kernel<kTiles, true>, grid, kLoThreads, 0, s, a, v, splits, per * kStep)
                : launch_dependent(expand_kernel<kTiles, false>, grid, kLoThreads, 0, s, a, v, splits, per * kStep);
}

} // namespace

// Ranges of k: one where the tiles fill the GPU, else about four CTAs an SM, each
// warp at least two blocks of columns.  (Two an SM: 16 us instead of 11 for 64 rows
// of 33 adapters, 16384 columns at rank 32; two ranges of 261 tiles cost 2 us more
// than one.)
int lora_splits(int n_rows, int k, int n_adapters, int sms)
{
    const int tiles = most_tiles(n_rows, n_adapters, kShrinkRows);
    int want = tiles >= sms ? 1 : 4 * sms / (tiles > 0 ? tiles : 1);
    const int most = (k + 31) / 32 / (2 * kLoWarps);
    want = want < most ? want : most;
    return want < 1 ? 1 : want;
}

// Rows of sums: splits * tiles is at most 4 sms, and tiles at least n_rows / 16, so
// splits * n_rows is at most 16 * 4 sms, or there is one range; with tiles of 128,
// at most sms tiles times ranges, or one range.
size_t lora_ws_bytes(int n_rows, int rank, int sms)
{
    const int64_t most = kTcPos * int64_t(sms), parts = int64_t(n_rows) > most ? int64_t(n_rows) : most;
    return align256(size_t(parts) * size_t(16 * rank_tiles(rank)) * sizeof(float));
}

cudaError_t lora_status(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_lora_status, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_lora_status, &zero, sizeof(int));
    }
    return e;
}

cudaError_t launch_lora(const w8_lora &a, float *v, int sms, cudaStream_t s)
{
    const cudaError_t e = raise_all();
    if (e != cudaSuccess)
        return e;
    switch (rank_tiles(a.rank)) {
    case 1: return lora<1>(a, v, sms, s);
    case 2: return lora<2>(a, v, sms, s);
    case 4: return lora<4>(a, v, sms, s);
    default: return lora<8>(a, v, sms, s);
    }
}

} // namespace w8
