// w8_latent_paged.cu -- latent attention, absorbed form, over the paged cache
// (w8_latent_attn_paged).
//
// With the rows of a group (query token, head) n, cached tokens j, latent
// columns d and a running reference m_n:
//   x_nj = q_n . [c_j | e_j],  p_nj = 2^(s x_nj - m_n),  s = scale log2 e
//   z_n = sum_j p_nj,  O_dn = sum_j c_jd p_nj,
//   out_n = O_.n / z_n,  lse_n = (m_n + log2 z_n) ln 2.
// All heads share the cached rows, so one copy of a tile of 64 tokens (72 KB)
// serves both products for up to 64 rows.  With 64 heads that is 121 flops a
// byte, under half of what the tensor cores do at the memory's rate: the
// kernel is bound by HBM there, and by latency when there is little to read.
//
// Both products run on tcgen05 with the accumulators in tensor memory:
//   S [64 rows x 64 tokens] = Q [64 x 576] * tile^T       (36 steps, M = 64)
//   O [128 d x NR rows] += tile[:, 128 d]^T * P^T [64 x NR]  (4 blocks x 4
//     steps, M = 128): the output is held transposed, d along the lanes, so
//     that its 512 x NR values take 4 NR columns -- with the rows along the
//     lanes it would fill all 512 columns and leave none for S -- and a group
//     of few rows costs few columns, not padding to 128.
// The tile lies in shared memory once, as 9 chunks of 64 columns in the
// 128-byte swizzle: K-major for the first product, and the same bytes
// MN-major for the second.  Rows of Q past the group read whatever follows
// in shared memory: they make rows of S that nobody reads.
//
// Twelve warps: 0-7 softmax and output (16 rows a warp, half the tile's tokens;
// S is read, the weights made against the reference as it stands, stored as bf16
// in shared memory, and redone when some row has passed its reference), 8 copies
// (tensor-map boxes of min(page, 64) tokens x 64 columns), 9 and 10 issue the two
// products (a warp each, so that a tile's second product does not wait for the
// next tile's copies), 11 loads the queries.  Two tiles are in flight, each in
// two halves: columns 0 .. 255, freed when the second product has passed over
// them, and the rest.  The next group's queries are loaded and scored while this
// one's output is stored.
// The reference moves only when a row's maximum passes it by 2^8 (p stays
// below 2^8, and 2^8 of fp32's range costs no precision): O is then rescaled
// in tensor memory, for most inputs once or twice in the first tiles.
//
// The work is cut by tiles, not by requests: all groups' tiles in one line,
// an equal run a CTA, one CTA an SM.  A group's begin takes two places of the
// line too, for the step from one group to the next costs a CTA about as much as
// two tiles (with no, one, two and four such places, 64 heads: 24 requests of 1
// to 4 query tokens 75.5, 73.0, 72.4, 73.4 us; 400 requests of up to 2000 tokens
// 121.6, 116.0, 109.7, 110.1; 16 heads, two and four: 89.7, 91.7); cuts that
// fall there move to the group's first tile, and split no group.  A group that
// more than one run touches leaves its parts (O, m, z in fp32) in the
// workspace, and a second kernel joins them.  Lengths are read on the device;
// the line's length picks NR: 64 rows a group, or fewer when there are not
// enough tiles to give every SM one.
//
// Measured (replayed, 64 heads): 128 requests of up to 16384 tokens, 0.99 million
// in all, 197 to 200 us for 1.16 GB (170 us at the rate of a copy), 6.1 TB/s in the
// first kernel, 1.10 million 221 us (190); 24 requests of 1 to 4 query tokens over up
// to 8111 tokens 66 to 73 us, bound by the chain copy - scores - softmax - output with
// two tiles in flight (2900 cycles a tile, the tensor cores' share 1920) and by the
// parts (26 MB written and read back); one request of 1531 tokens 13 us, latency.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "w8_copies.h"
#include "w8_device.cuh"
#include "w8_serve_internal.h"
#include "w8_tcgen.cuh"

namespace w8 {

__device__ int g_paged_status;

namespace {

using namespace tcg;

constexpr int kTile = 64;                    // tokens
constexpr int kChunk = kTile * 128;          // bytes of 64 tokens x 64 columns
constexpr int kFront = 4, kBack = 5;         // chunks of a tile's two halves: columns 0 .. 255, 256 .. 575
constexpr int kMaxRows = 64;
constexpr int kPagedThreads = 384, kSoftThreads = 256, kCopyWarp = 8, kScoreWarp = 9, kOutWarp = 10, kQueryWarp = 11;
constexpr int kMaxSlots = 3;
constexpr int kSmem = 227 * 1024 - 2048;     // what the CTA takes; the rest is static
constexpr int kTmemCols = 512;
constexpr int kSeveral = 128;                // above any count of rows, see paged_kernel
constexpr int kBegin = 2;                    // places of a group's begin in the line
constexpr float kRaise = 8.0f;               // log2 of how far a row's weights may pass 1
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Shared memory for groups of nr rows: Q, P, then the two halves' rings.
struct Smem {
    int q, p, front, back, fronts, backs, end;
};
__host__ __device__ constexpr Smem smem_plan(int nr)
{
    Smem s{};
    s.q = 0;
    s.p = s.q + 9 * nr * 128;
    s.front = s.p + nr * 128;
    s.fronts = nr == 64 ? 2 : 3;
    s.back = s.front + s.fronts * kFront * kChunk;
    s.backs = 2;
    s.end = s.back + s.backs * kBack * kChunk;
    return s;
}
static_assert(smem_plan(64).end <= kSmem - 1024 && smem_plan(32).end <= kSmem - 1024 && smem_plan(16).end <= kSmem - 1024,
              "shared memory");
// the first product reads 64 rows from every chunk of Q: the last chunk's
// reach past Q stays inside the allocation
static_assert(smem_plan(16).end >= 8 * 16 * 128 + kChunk, "Q's reach");

// What the parts of split groups need: [2 CTAs][64][512] fp32, [2 CTAs][64]
// (m, z), [CTAs] the group that runs over the CTA's start, if it runs over no
// earlier CTA's.
struct Boundary {
    int first, last; // CTAs that hold the group's parts; last < 0: this CTA's start is no group's first crossed one
    int row0, rows;  // the group's rows, counted over all query tokens' heads
};
struct Parts {
    float *o;
    float2 *mz;
    Boundary *at;
};
__host__ __device__ inline size_t parts_bytes(int ctas)
{
    return size_t(ctas) * (2 * kMaxRows * (W8_LATENT_DIM * 4 + 8) + sizeof(Boundary)) + 256;
}
__host__ __device__ inline Parts parts_of(void *ws, int ctas)
{
    Parts p;
    p.o = static_cast<float *>(ws);
    p.mz = reinterpret_cast<float2 *>(p.o + size_t(ctas) * 2 * kMaxRows * W8_LATENT_DIM);
    p.at = reinterpret_cast<Boundary *>(p.mz + size_t(ctas) * 2 * kMaxRows);
    return p;
}

struct Request {
    int q0, q, len; // first query token, query tokens, cached tokens
};
__device__ __forceinline__ Request request_of(const w8_latent_paged &a, int r)
{
    Request q;
    q.q0 = min(max(__ldg(a.cu_q + r), 0), a.n_tok);
    q.q = min(max(__ldg(a.cu_q + r + 1), q.q0), a.n_tok) - q.q0;
    const int64_t cap = int64_t(a.max_pages) * a.cache.page_size;
    q.len = int(min(int64_t(max(__ldg(a.seq_lens + r), 0)), min(cap, int64_t(0x7FFFFF00))));
    return q;
}
// Cached tokens that query token i of the request sees.
__device__ __forceinline__ int seen(const Request &q, int i)
{
    const int64_t n = int64_t(q.len) - q.q + i + 1;
    return int(n < 0 ? 0 : n > q.len ? q.len : n);
}
// The query token of a row of the request; most requests have one.
__device__ __forceinline__ int token_of(const Request &q, int heads, int row) { return q.q == 1 ? 0 : row / heads; }
// Cached tokens that the last row of group g sees.
__device__ __forceinline__ int group_sees(const Request &q, int heads, int nr, int g)
{
    return seen(q, token_of(q, heads, min((g + 1) * nr, q.q * heads) - 1));
}
// Their tiles, one (of nothing) if there are none.
__device__ __forceinline__ int tiles_of_sees(int vis) { return vis < 1 ? 1 : (vis + kTile - 1) / kTile; }
__device__ __forceinline__ int groups_of(const Request &q, int heads, int nr) { return (q.q * heads + nr - 1) / nr; }

// One CTA's place in the line, a run of one group at a time.  Every role walks
// it for itself.  A group takes kBegin places and one for each of its tiles.
struct Walk {
    int64_t pos, end;  // the next tile's place, the CTA's last + 1
    int r, g, off;     // its request, group, place in the group
    Request req;
    int vis, tiles;    // what the group's last row sees
    int run;           // tiles of this run

    __device__ __forceinline__ bool next(const w8_latent_paged &a, int nr, bool first)
    {
        if (!first) { // the first request comes with the place
            pos += run + kBegin;
            off = 0;
            if (pos < end && ++g >= groups_of(req, a.n_heads, nr)) {
                g = 0;
                do
                    req = request_of(a, ++r);
                while (req.q == 0 && r + 1 < a.n_req);
            }
        }
        if (pos >= end)
            return false;
        vis = group_sees(req, a.n_heads, nr, g);
        tiles = tiles_of_sees(vis);
        run = int(min(int64_t(tiles - off), end - pos));
        return true;
    }
};

// 2 KB at most: the rest is the rings'.
struct Shared {
    uint64_t front_full[kMaxSlots], front_free[kMaxSlots], back_full[kMaxSlots], back_free[kMaxSlots];
    uint64_t q, q_free, s[2], s_free[2], p, o, end[2];
    int64_t out[kMaxRows]; // a row's place in the output
    int64_t sum[kPagedThreads / 32];
    int max[kPagedThreads / 32], few[kPagedThreads / 32];
    int start[4];
    Request req;
    uint32_t tmem;
    float f[kMaxRows], top[2][kMaxRows];
};

static_assert(sizeof(Shared) <= 227 * 1024 - kSmem, "shared memory");

// A ring's next slot and the parity of its use.
struct Turn {
    int k = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void step(int slots)
    {
        if (++k == slots) {
            k = 0;
            parity ^= 1;
        }
    }
};

// ---- copies ---------------------------------------------------------------
// One lane does it all: two waits, two byte counts and 9 BOXES copies a tile.
// (The loop must be short: with four half-size units a tile, votes and a
// shared loop body it took 2500 cycles a tile, near the tile's share of HBM.)
template <int NR, int BOXES>
__device__ __forceinline__ bool copy_loop(const w8_latent_paged &a, const CUtensorMap &map, Walk w, uint8_t *sm, Shared &sh, uint64_t policy)
{
    constexpr Smem lay = smem_plan(NR);
    constexpr int kBox = kTile / BOXES;
    const int page = a.cache.page_size, shift = 31 - __clz(page);
    const uint32_t front = smem_addr(sm + lay.front), back = smem_addr(sm + lay.back);
    Ring<lay.fronts> f;
    Ring<lay.backs> b;
    bool ok = true;
    for (bool first = true; ok && w.next(a, NR, first); first = false) {
        const int32_t *table = a.block_table + int64_t(w.r) * a.ld_table;
        const int vis = w.vis;
        const int end = vis > 0 ? w.off + w.run : w.off; // a group that sees nothing has a tile of nothing
        int pages[BOXES], ahead[BOXES]; // the next tile's pages are fetched ahead
        auto fetch = [&](int (&pg)[BOXES], int t) {
#pragma unroll
            for (int i = 0; i < BOXES; ++i) {
                const int j = t * kTile + i * kBox;
                pg[i] = t < end && j < vis ? __ldg(table + (j >> shift)) : 0;
            }
        };
        fetch(pages, w.off);
        for (int t = w.off; t < end; ++t) {
            fetch(ahead, t + 1);
            const int left = min(vis - t * kTile, kTile);
            const int need = (left + kBox - 1) / kBox;            // boxes with a key that is seen
            const int y = BOXES == 1 ? t * kTile & (page - 1) : 0; // a page of several tiles
#pragma unroll
            for (int i = 0; i < BOXES; ++i) // a number that is no page reads as zeros
                pages[i] = pages[i] < 0 || pages[i] > a.cache.n_pages ? a.cache.n_pages : pages[i];
            ok = f.take([&](int k, uint32_t parity) { return bar_wait(&sh.front_free[k], parity); });
            if (!ok)
                break;
            bar_expect(&sh.front_full[f.k], uint32_t(kFront * kBox * 128) * need);
#pragma unroll
            for (int c = 0; c < kFront; ++c)
#pragma unroll
                for (int i = 0; i < BOXES; ++i)
                    if (i < need)
                        copy_box(front + uint32_t(f.k * kFront * kChunk + c * kChunk + i * kBox * 128), &map, 64 * c, y, pages[i],
                                 &sh.front_full[f.k], policy);
            f.filled();
            ok = b.take([&](int k, uint32_t parity) { return bar_wait(&sh.back_free[k], parity); });
            if (!ok)
                break;
            bar_expect(&sh.back_full[b.k], uint32_t(kBack * kBox * 128) * need);
#pragma unroll
            for (int c = 0; c < kBack; ++c)
#pragma unroll
                for (int i = 0; i < BOXES; ++i)
                    if (i < need)
                        copy_box(back + uint32_t(b.k * kBack * kChunk + c * kChunk + i * kBox * 128), &map, 64 * (kFront + c), y,
                                 pages[i], &sh.back_full[b.k], policy);
            b.filled();
#pragma unroll
            for (int i = 0; i < BOXES; ++i)
                pages[i] = ahead[i];
        }
    }
    // the copies still in flight (there are any only after a wait elsewhere gave up)
    f.drain([&](int k, uint32_t parity) { bar_wait(&sh.front_full[k], parity); });
    b.drain([&](int k, uint32_t parity) { bar_wait(&sh.back_full[k], parity); });
    return ok;
}
template <int NR>
__device__ __forceinline__ bool copy_role(const w8_latent_paged &a, const CUtensorMap &map, const Walk &w, uint8_t *sm, Shared &sh, bool once)
{
    bool ok = true;
    if (elect_one()) {
        // rows that one group reads leave L2 first: the parts of split groups stay
        const uint64_t policy = once ? policy_first() : policy_normal();
        ok = a.cache.page_size == 16   ? copy_loop<NR, 4>(a, map, w, sm, sh, policy)
             : a.cache.page_size == 32 ? copy_loop<NR, 2>(a, map, w, sm, sh, policy)
                                       : copy_loop<NR, 1>(a, map, w, sm, sh, policy);
    }
    __syncwarp();
    return ok;
}

// ---- first product ----------------------------------------------------------
template <int NR>
__device__ __forceinline__ bool score_role(const w8_latent_paged &a, Walk w, uint8_t *sm, Shared &sh, uint32_t tm_s)
{
    constexpr Smem lay = smem_plan(NR);
    constexpr uint32_t id = inst_desc(64, kTile, false, false);
    const uint64_t dq = desc128_k(smem_addr(sm + lay.q), 1024);
    const uint64_t dfront = desc128_k(smem_addr(sm + lay.front), 1024), dback = desc128_k(smem_addr(sm + lay.back), 1024);
    const bool one = elect_one();
    Turn f, b;
    int runs = 0, n = 0; // runs with keys, tiles
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) { ok = __all_sync(0xffffffffu, ok && bar_wait(bar, parity & 1)); };
    for (bool first = true; ok && w.next(a, NR, first); first = false) {
        if (w.vis == 0)
            continue;
        wait(&sh.q, uint32_t(runs));
        ++runs;
        for (int t = 0; ok && t < w.run; ++t, ++n) {
            // S of tile n - 2, in the same columns, has been read
            if (n >= 2)
                wait(&sh.s_free[n & 1], uint32_t(n / 2 - 1));
            const uint32_t d = tm_s + uint32_t(n & 1) * kTile;
            wait(&sh.front_full[f.k], f.parity);
            if (!ok)
                break;
            fence_after();
            const uint64_t df = dfront + uint64_t((f.k * kFront * kChunk) >> 4);
            if (one) {
#pragma unroll
                for (int s = 0; s < 4 * kFront; ++s)
                    mma_ss(d, dq + uint64_t(((s / 4) * NR * 128 + (s % 4) * 32) >> 4),
                           df + uint64_t(((s / 4) * kChunk + (s % 4) * 32) >> 4), id, uint32_t(s));
            }
            __syncwarp();
            f.step(lay.fronts);
            wait(&sh.back_full[b.k], b.parity);
            if (!ok)
                break;
            fence_after();
            const uint64_t db = dback + uint64_t((b.k * kBack * kChunk) >> 4);
            if (one) {
#pragma unroll
                for (int s = 0; s < 4 * kBack; ++s)
                    mma_ss(d, dq + uint64_t(((kFront + s / 4) * NR * 128 + (s % 4) * 32) >> 4),
                           db + uint64_t(((s / 4) * kChunk + (s % 4) * 32) >> 4), id, 1);
                commit(&sh.s[n & 1]);
                if (t == w.run - 1)
                    commit(&sh.q_free);
            }
            __syncwarp();
            b.step(lay.backs);
        }
    }
    // nothing of this warp's is in the tensor cores when the CTA frees its memory
    if (one)
        commit(&sh.end[0]);
    __syncwarp();
    return bar_wait(&sh.end[0], 0) && ok;
}

// ---- second product ---------------------------------------------------------
template <int NR>
__device__ __forceinline__ bool out_role(const w8_latent_paged &a, Walk w, uint8_t *sm, Shared &sh, uint32_t tmem)
{
    constexpr Smem lay = smem_plan(NR);
    constexpr uint32_t id = inst_desc(128, NR, true, false);
    const uint64_t dp = desc128_k(smem_addr(sm + lay.p), 1024), dfront = desc128(smem_addr(sm + lay.front), kChunk, 1024),
                   dback = desc128(smem_addr(sm + lay.back), kChunk, 1024);
    const bool one = elect_one();
    Turn f, b;
    int n = 0;
    bool ok = true;
    for (bool first = true; ok && w.next(a, NR, first); first = false) {
        if (w.vis == 0)
            continue;
        for (int t = 0; ok && t < w.run; ++t, ++n) {
            ok = __all_sync(0xffffffffu, bar_wait(&sh.p, uint32_t(n & 1)));
            if (!ok)
                break;
            fence_after();
            const uint64_t df = dfront + uint64_t((f.k * kFront * kChunk) >> 4), db = dback + uint64_t((b.k * kBack * kChunk) >> 4);
            if (one) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        mma_ss(tmem + uint32_t(u * NR), (u < 2 ? df : db) + uint64_t(((u % 2) * 2 * kChunk + s * 2048) >> 4),
                               dp + uint64_t((s * 32) >> 4), id, uint32_t(t | s));
                    if (u == 1)
                        commit(&sh.front_free[f.k]);
                }
                commit(&sh.back_free[b.k]);
                commit(&sh.o);
            }
            __syncwarp();
            f.step(lay.fronts);
            b.step(lay.backs);
        }
    }
    if (one)
        commit(&sh.end[1]);
    __syncwarp();
    return bar_wait(&sh.end[1], 0) && ok;
}

// ---- queries ----------------------------------------------------------------
// Q of each run, by a warp of its own: the next run's is on its way while this
// one's output is stored.  8 lanes take 128 bytes of a row, 4 rows a step; rows
// past the group's are zeros.
template <int NR>
__device__ __forceinline__ bool query_role(const w8_latent_paged &a, Walk w, uint8_t *sm, Shared &sh, int lane)
{
    constexpr Smem lay = smem_plan(NR);
    const uint32_t q = smem_addr(sm + lay.q);
    const int v = lane & 7;
    int runs = 0; // with keys
    bool ok = true;
    for (bool first = true; ok && w.next(a, NR, first); first = false) {
        if (w.vis == 0)
            continue;
        // the last run's scores are made
        if (runs > 0)
            ok = __all_sync(0xffffffffu, bar_wait(&sh.q_free, uint32_t((runs - 1) & 1)));
        if (!ok)
            break;
        ++runs;
        const int row0 = w.g * NR, rows = min(NR, w.req.q * a.n_heads - row0);
        int row = lane >> 3, tok = token_of(w.req, a.n_heads, row0 + row), head = row0 + row - tok * a.n_heads;
#pragma unroll 2
        for (; row < NR; row += 4) {
            const bool some = row < rows;
            const uint16_t *lat = some ? a.q_lat + (w.req.q0 + tok) * a.ld_qlat_tok + head * a.ld_qlat_head + 8 * v : a.q_lat;
            const uint16_t *rope = some ? a.q_rope + (w.req.q0 + tok) * a.ld_qrope_tok + head * a.ld_qrope_head + 8 * v : a.q_rope;
            const uint32_t to = q + row * 128 + ((v ^ (row & 7)) << 4);
#pragma unroll
            for (int c = 0; c < 9; ++c)
                copy16(to + c * NR * 128, c < 8 ? lat + 64 * c : rope, some);
            for (head += 4; head >= a.n_heads; head -= a.n_heads)
                ++tok;
        }
        copy16_wait();
        fence_async_shared();
        bar_arrive(&sh.q);
    }
    return ok;
}

// ---- softmax, output --------------------------------------------------------
// A pair of bf16 values with zeros for those that are not finite.
__device__ __forceinline__ uint32_t finite2(uint32_t u)
{
    u = (u & 0x7F80u) == 0x7F80u ? u & 0xFFFF0000u : u;
    return (u & 0x7F800000u) == 0x7F800000u ? u & 0xFFFFu : u;
}
// Zeros for values that are not finite in rows `from` .. of a tile's latents, `vecs`
// 16-byte vectors a chunk, once the two halves are here: 1 if there were any among
// this thread's, -1 if a wait gave up.
__device__ __noinline__ int clear_hidden(uint64_t *front_full, uint32_t front_parity, uint8_t *front, uint64_t *back_full,
                                         uint32_t back_parity, uint8_t *back, int from, int vecs, int tid)
{
    if (!bar_wait(front_full, front_parity) || !bar_wait(back_full, back_parity))
        return -1;
    int found = 0;
    for (int i = tid; i < 8 * vecs; i += kSoftThreads) {
        const int c = i / vecs, rest = i - c * vecs;
        uint4 *at = reinterpret_cast<uint4 *>((c < kFront ? front + c * kChunk : back + (c - kFront) * kChunk) + from * 128 + rest * 16);
        const uint4 u = *at, v = make_uint4(finite2(u.x), finite2(u.y), finite2(u.z), finite2(u.w));
        if (u.x != v.x || u.y != v.y || u.z != v.z || u.w != v.w) {
            *at = v;
            found = 1;
        }
    }
    return found;
}
// NaN in the outputs of a run's rows (row0 .., `rows` of them) that see a value that
// is not finite in the request's tokens from .. to - 1: in `out` at the rows' places,
// or in the run's part.
__device__ __noinline__ void poison(const w8_latent_paged &a, int r, int row0, int rows, int from, int to, const int64_t *places,
                                    float *part, int tid)
{
    const Request q = request_of(a, r);
    const int page = a.cache.page_size, shift = 31 - __clz(page);
    for (int j = from; j < to; ++j) {
        const int p = __ldg(a.block_table + r * a.ld_table + (j >> shift));
        if (p < 0 || p >= a.cache.n_pages) // reads as zeros
            continue;
        const uint16_t *at = static_cast<const uint16_t *>(a.cache.data) + p * a.cache.ld_page + (j & (page - 1)) * a.cache.ld_tok;
        for (int d = tid; d < W8_LATENT_DIM; d += kSoftThreads)
            if ((__ldg(at + d) & 0x7F80u) == 0x7F80u)
                for (int i = 0; i < rows; ++i)
                    if (j < seen(q, token_of(q, a.n_heads, row0 + i))) {
                        if (part)
                            part[i * W8_LATENT_DIM + d] = CUDART_NAN_F;
                        else
                            a.out[places[i] + d] = 0x7FFF;
                    }
    }
}
// kMixed: groups may hold rows of several query tokens, which do not see the same.
// (Code of its own, since it slows a tile: 24 requests of 1 to 4 query tokens at 64
// heads, whose groups are never mixed, 74.6 us with it against 72.4.)
template <int NR, bool kMixed>
__device__ __forceinline__ bool softmax_role(const w8_latent_paged &a, Walk w, uint8_t *sm, Shared &sh, uint32_t tmem,
                                             uint32_t tm_s, const Parts &parts, int64_t total, int64_t ctas, int tid)
{
    constexpr Smem lay = smem_plan(NR);
    const int warp = tid >> 5, lane = tid & 31;
    // warps w and w + 4 share 16 rows: tokens 0 .. 31 and 32 .. 63 of the tile
    const int quarter = warp & 3, half = warp >> 2;
    const float sl = a.scale * kLog2e;
    const int g4 = lane >> 2, t4 = lane & 3;
    const bool active = 16 * quarter < NR; // warps that have rows
    const uint32_t lanes = uint32_t(32 * quarter) << 16;
    const int row_h[2] = {16 * quarter + g4, 16 * quarter + g4 + 8}; // this thread's rows
    bool ok = true;
    // a wait that gave up is followed by no other, but every barrier below is
    // still met, so that no warp waits for one that left
    auto wait = [&](uint64_t *bar, int phase) { ok = __all_sync(0xffffffffu, ok && bar_wait(bar, uint32_t(phase & 1))); };
    if (tid == 0 && (w.pos >= w.end || w.off == 0))
        parts.at[blockIdx.x].last = -1; // no group runs over this CTA's start
    int n = 0; // tiles so far
    for (bool have = w.next(a, NR, true); have;) {
        const int row0 = w.g * NR, rows = min(NR, w.req.q * a.n_heads - row0);
        const int vis = w.vis;
        // Tokens from here on are hidden from some of the group's rows (of earlier
        // query tokens).  Their weights there are 0, and 0 x NaN is not: values that
        // are not finite are made zero for the second product, and the output of the
        // rows that do see them is made NaN in the end.
        int hidden = INT32_MAX;
        if (kMixed && w.req.q > 1) {
            const int lo = seen(w.req, token_of(w.req, a.n_heads, row0));
            hidden = lo < vis ? lo : INT32_MAX;
        }
        bool found = false;
        // how many keys this thread's rows see
        int lim[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            lim[h] = row_h[h] < rows ? seen(w.req, token_of(w.req, a.n_heads, row0 + row_h[h])) : 0;
        if (tid < rows) {
            const int tok = token_of(w.req, a.n_heads, row0 + tid), head = row0 + tid - tok * a.n_heads;
            sh.out[tid] = (w.req.q0 + tok) * a.ld_out_tok + head * a.ld_out_head;
        }
        if (w.off > 0 && tid == 0) {
            // the group runs over this CTA's start
            const int64_t s0 = w.pos - w.off, s1 = s0 + w.tiles - 1; // the group's tiles' places
            Boundary b;
            b.first = int(((s0 + 1) * ctas - 1) / total);
            b.last = int(((s1 + 1) * ctas - 1) / total);
            b.row0 = w.req.q0 * a.n_heads + row0;
            b.rows = rows;
            if (b.first != int(blockIdx.x) - 1)
                b.last = -1; // an earlier start names the group
            parts.at[blockIdx.x] = b;
        }
        // the run after this one, looked up while the first tile's output is summed
        Walk nx = w;
        bool more = false;
        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, z[2] = {0.0f, 0.0f};
        if (vis == 0)
            more = nx.next(a, NR, false);
        if (vis > 0) {
            for (int t = 0; t < w.run; ++t, ++n) {
                const int j0 = (w.off + t) * kTile, c0 = j0 + 32 * half; // tile's, thread's first token
                wait(&sh.s[n & 1], n >> 1);
                fence_after();
                float x[16];
                if (active) {
                    ld16x32(x, tm_s + lanes + uint32_t((n & 1) * kTile + 32 * half));
                    wait_ld();
                }
                fence_before();
                bar_arrive(&sh.s_free[n & 1]);
                // Weights against the reference as it stands; whether any row has
                // passed it is asked afterwards, so that no exponential waits
                // for a maximum.
                uint32_t p[2][4];
                float sum[2];
                auto weigh = [&](int h) {
                    const float ref = m[h] == -CUDART_INF_F ? 0.0f : m[h];
                    float e[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        e[i] = ex2(fmaf(x[4 * (i >> 1) + 2 * h + (i & 1)], sl, -ref));
                    sum[h] = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        p[h][j] = pack_bf16(e[2 * j], e[2 * j + 1]);
                };
                auto store_p = [&] {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint8_t *to = sm + lay.p + row_h[h] * 128 + 4 * t4;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint32_t *>(to + (((4 * half + j) ^ (row_h[h] & 7)) << 4)) = p[h][j];
                    }
                };
                float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
                bool raise = false;
                if (active) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (c0 + 32 > lim[h]) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (c0 + 8 * (i >> 1) + 2 * t4 + (i & 1) >= lim[h])
                                    x[4 * (i >> 1) + 2 * h + (i & 1)] = -CUDART_INF_F;
                        }
                        if (t > 0) // the first tile's reference is not known yet
                            weigh(h);
                        float top[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            top[j] = fmaxf(x[4 * j + 2 * h], x[4 * j + 2 * h + 1]);
                        mx[h] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sl;
                        // -inf + 8 is -inf: the first key that is seen raises it
                        raise = raise || mx[h] > m[h] + kRaise;
                    }
                }
                // the last tile's second product has read P and written O
                if (t > 0) {
                    wait(&sh.o, n - 1);
                    if (active)
                        store_p();
                }
                if (kMixed && j0 + kTile > hidden) {
                    // (the copies are waited for once more: these threads read them themselves)
                    const int from = max(hidden - j0, 0), f = n % lay.fronts, b = n % lay.backs;
                    const int got = clear_hidden(&sh.front_full[f], n / lay.fronts & 1, sm + lay.front + f * kFront * kChunk,
                                                 &sh.back_full[b], n / lay.backs & 1, sm + lay.back + b * kBack * kChunk, from,
                                                 8 * (min(vis - j0, kTile) - from), tid);
                    found = found || got > 0;
                    ok = __all_sync(0xffffffffu, ok && got >= 0);
                }
                if (j0 + kTile > vis) {
                    // rows of the tile that nobody sees may hold anything: their weights are 0, 0 x NaN is not
                    const int dead = kTile - (vis - j0);
                    for (int i = tid; i < dead * 64; i += kSoftThreads) {
                        const int c = i / (dead * 8), rest = i - c * dead * 8;
                        uint8_t *to = c < kFront ? sm + lay.front + (n % lay.fronts * kFront + c) * kChunk
                                                 : sm + lay.back + (n % lay.backs * kBack + c - kFront) * kChunk;
                        *reinterpret_cast<uint4 *>(to + (vis - j0) * 128 + rest * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                if (sync_any(1, kSoftThreads, raise || t == 0)) {
                    // the rows' maxima over both halves, the new references, the weights again
                    if (active) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                            if (t4 == 0)
                                sh.top[half][row_h[h]] = mx[h];
                        }
                    }
                    sync_some(1, kSoftThreads);
                    if (active) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float all = fmaxf(sh.top[0][row_h[h]], sh.top[1][row_h[h]]);
                            float f = 1.0f;
                            if (t == 0) {
                                m[h] = all;
                            } else if (all > m[h] + kRaise) { // from -inf: nothing is summed yet, f is 0
                                f = ex2(m[h] - all);
                                m[h] = all;
                                z[h] *= f;
                            }
                            weigh(h);
                            if (t4 == 0 && half == 0)
                                sh.f[row_h[h]] = f;
                        }
                        store_p();
                    }
                    sync_some(1, kSoftThreads);
                    if (t > 0) {
                        fence_after();
#pragma unroll 1
                        for (int c = half; c < NR / 4; c += 2) { // 16 columns: rows 16 c % NR .. of block 16 c / NR
                            float o[16];
                            ld32x16(o, tmem + lanes + uint32_t(16 * c));
                            wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] *= sh.f[(16 * c) % NR + i];
                            st32x16(tmem + lanes + uint32_t(16 * c), o);
                        }
                        wait_st();
                    }
                }
                if (active) {
                    z[0] += sum[0];
                    z[1] += sum[1];
                }
                fence_before();
                fence_async_shared();
                bar_arrive(&sh.p);
                if (t == 0)
                    more = nx.next(a, NR, false);
            }
        }
        // ---- the run's result: the output, or a part of it
        const bool whole = w.off == 0 && w.run == w.tiles;
        const int slot = 2 * int(blockIdx.x) + (w.off == 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            z[h] += __shfl_xor_sync(0xffffffffu, z[h], 1);
            z[h] += __shfl_xor_sync(0xffffffffu, z[h], 2);
            if (active && t4 == 0 && half == 1)
                sh.top[1][row_h[h]] = z[h];
        }
        bool poisoned = false;
        if constexpr (kMixed)
            poisoned = sync_any(1, kSoftThreads, found);
        else
            sync_some(1, kSoftThreads);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = row_h[h];
            if (active && t4 == 0 && half == 0) {
                const float zz = z[h] + sh.top[1][row];
                const bool some = zz > 0.0f || zz != zz;
                sh.f[row] = some ? 1.0f / zz : 0.0f;
                if (row < rows) {
                    if (!whole)
                        parts.mz[slot * kMaxRows + row] = make_float2(m[h], zz);
                    else if (a.lse)
                        a.lse[int64_t(w.req.q0) * a.n_heads + row0 + row] = some ? (m[h] + log2f(zz)) * kLn2 : -CUDART_INF_F;
                }
            }
        }
        if (vis > 0)
            wait(&sh.o, n - 1);
        fence_after();
        sync_some(1, kSoftThreads);
        // warp halves take alternate runs of 16 rows, two runs' loads at a time
        constexpr int kRuns = NR / 8; // of a warp
#pragma unroll 1
        for (int c0 = 0; c0 < kRuns; c0 += 2) {
            float o[2][16];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (vis > 0)
                    ld32x16(o[k], tmem + lanes + uint32_t(16 * (2 * (c0 + k) + half)));
            wait_ld();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = 2 * (c0 + k) + half, n0 = (16 * c) % NR, d0 = 128 * (16 * c / NR) + 32 * quarter;
                if (n0 >= rows)
                    continue;
                if (whole) {
                    // lane pairs trade halves, so that each stores two columns of one row; all
                    // is ready before the first store, behind which no shared load may move
                    uint32_t two[8];
                    uint16_t *to[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float e = vis > 0 ? o[k][2 * i] * sh.f[n0 + 2 * i] : 0.0f,
                                    d = vis > 0 ? o[k][2 * i + 1] * sh.f[n0 + 2 * i + 1] : 0.0f;
                        const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? e : d, 1);
                        two[i] = lane & 1 ? pack_bf16(got, d) : pack_bf16(e, got);
                        to[i] = a.out + sh.out[n0 + 2 * i + (lane & 1)] + d0 + (lane & ~1);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (n0 + 2 * i + (lane & 1) < rows)
                            *reinterpret_cast<uint32_t *>(to[i]) = two[i];
                } else {
                    float *to = parts.o + (size_t(slot) * kMaxRows + n0) * W8_LATENT_DIM + d0 + lane;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (n0 + i < rows)
                            to[i * W8_LATENT_DIM] = o[k][i];
                }
            }
        }
        fence_before(); // the loads of O, before the next run's products
        sync_some(1, kSoftThreads); // the rows' places and 1 / z are read
        if (kMixed && poisoned) {
            poison(a, w.r, row0, rows, max(hidden, w.off * kTile), int(min(int64_t(w.off + w.run) * kTile, int64_t(vis))), sh.out,
                   whole ? nullptr : parts.o + size_t(slot) * kMaxRows * W8_LATENT_DIM, tid);
            sync_some(1, kSoftThreads);
        }
        w = nx;
        have = more;
    }
    return ok;
}

__global__ void __launch_bounds__(kPagedThreads, 1)
    paged_kernel(const __grid_constant__ w8_latent_paged a, const __grid_constant__ CUtensorMap map, void *ws)
{
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ __align__(16) Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *const sm = s_dyn + ((1024u - (smem_addr(s_dyn) & 1023u)) & 1023u);
    if (tid == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            bar_init(&sh.front_full[i], 1);
            bar_init(&sh.front_free[i], 1);
            bar_init(&sh.back_full[i], 1);
            bar_init(&sh.back_free[i], 1);
        }
        bar_init(&sh.q, 32);
        bar_init(&sh.q_free, 1);
        bar_init(&sh.s[0], 1);
        bar_init(&sh.s[1], 1);
        bar_init(&sh.s_free[0], kSoftThreads);
        bar_init(&sh.s_free[1], kSoftThreads);
        bar_init(&sh.p, kSoftThreads);
        bar_init(&sh.o, 1);
        bar_init(&sh.end[0], 1);
        bar_init(&sh.end[1], 1);
        bar_init_fence();
    }
    if (warp == 0)
        tmem_alloc(&sh.tmem, kTmemCols);
    pdl_wait();

    // ---- the line of tiles: NR, its length, this CTA's run -------------------
    const int per = (a.n_req + kPagedThreads - 1) / kPagedThreads;
    const int r0 = min(tid * per, a.n_req), r1 = min(r0 + per, a.n_req);
    Request held{0, 0, 0}; // the thread's first request, mostly its only one
    if (r0 < r1)
        held = request_of(a, r0);
    // this thread's tiles with nr rows a group, and a group's begin as that of so many
    auto tiles_of = [&](int nr, int begin) {
        int64_t sum = 0;
        for (int r = r0; r < r1; ++r) {
            const Request q = r == r0 ? held : request_of(a, r);
            const int n = groups_of(q, a.n_heads, nr);
            sum += int64_t(n) * begin;
            if (q.q == 1) // all groups see the same
                sum += int64_t(n) * max((q.len + kTile - 1) / kTile, 1);
            else
                for (int g = 0; g < n; ++g)
                    sum += tiles_of_sees(group_sees(q, a.n_heads, nr, g));
        }
        return sum;
    };
    int rows = 0, groups64 = 0;
    for (int r = r0; r < r1; ++r) {
        const Request q = r == r0 ? held : request_of(a, r);
        rows = max(rows, min(q.q * a.n_heads, kMaxRows + 1) + (q.q > 1 ? kSeveral : 0));
        groups64 += groups_of(q, a.n_heads, 64);
    }
    // fewer rows a group: when no group would be filled, or when twice as many
    // groups still leave no SM two tiles (a thread's count past 2^16 is many)
    rows = __reduce_max_sync(0xffffffffu, rows);
    int64_t mine = tiles_of(64, 0);
    const int few = __reduce_add_sync(0xffffffffu, int(min(mine, int64_t(1 << 16))));
    if (lane == 0) {
        sh.max[warp] = rows;
        sh.few[warp] = few;
    }
    __syncthreads();
    int all64 = 0;
    for (int i = 0; i < kPagedThreads / 32; ++i) {
        rows = max(rows, sh.max[i]);
        all64 += sh.few[i];
    }
    // (those of a request of several query tokens are the most there are)
    const bool several = rows >= kSeveral;
    rows -= several ? kSeveral : 0;
    const int grid = int(gridDim.x), rows_max = rows;
    const int nr = rows > 32 && all64 * 2 > grid ? 64 : rows > 16 && all64 * 4 > grid ? 32 : 16;
    mine = nr != 64 ? tiles_of(nr, kBegin) : mine + int64_t(groups64) * kBegin;
    int64_t inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
        inc += lane >= d ? o : 0;
    }
    if (lane == 31)
        sh.sum[warp] = inc;
    __syncthreads();
    int64_t before = inc - mine, total = 0;
    for (int i = 0; i < kPagedThreads / 32; ++i) {
        before += i < warp ? sh.sum[i] : 0;
        total += sh.sum[i];
    }
    const int64_t ctas = min(total, int64_t(gridDim.x)); // those that have work
    Walk w{};
    if (total * ctas < int64_t(1) << 32) { // 64-bit division is a call of some hundred instructions
        const uint32_t t = uint32_t(total), c = uint32_t(ctas);
        w.pos = c ? min(blockIdx.x, c) * t / c : 0;
        w.end = c ? min(blockIdx.x + 1, c) * t / c : 0;
    } else {
        w.pos = min(int64_t(blockIdx.x), ctas) * total / ctas;
        w.end = min(int64_t(blockIdx.x) + 1, ctas) * total / ctas;
    }
    if (w.pos < w.end && before <= w.pos && w.pos < before + mine) {
        int64_t at = before;
        for (int r = r0; r < r1; ++r) {
            const Request q = r == r0 ? held : request_of(a, r);
            const int n = groups_of(q, a.n_heads, nr);
            for (int g = 0; g < n; ++g) {
                const int t = kBegin + tiles_of_sees(group_sees(q, a.n_heads, nr, g));
                if (at <= w.pos && w.pos < at + t) {
                    const int place = int(w.pos - at);
                    sh.start[0] = r;
                    sh.start[1] = g;
                    sh.start[2] = max(place - kBegin, 0);
                    sh.start[3] = max(kBegin - place, 0);
                    sh.req = q;
                }
                at += t;
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem, tm_s = tmem + 4 * kMaxRows; // O in columns 0 .., S after it
    if (w.pos < w.end) { // else nobody has written the start
        w.r = sh.start[0];
        w.g = sh.start[1];
        w.off = sh.start[2];
        w.req = sh.req;
        w.pos += sh.start[3]; // past the group's begin; a CTA may have nothing else
    }
    const Parts parts = parts_of(ws, int(gridDim.x));
    const int role = __shfl_sync(0xffffffffu, warp, 0);
    auto roles = [&](auto rows) {
        constexpr int NR = decltype(rows)::value;
        return role == kCopyWarp    ? copy_role<NR>(a, map, w, sm, sh, rows_max <= NR)
               : role == kScoreWarp ? score_role<NR>(a, w, sm, sh, tm_s)
               : role == kOutWarp   ? out_role<NR>(a, w, sm, sh, tmem)
               : role == kQueryWarp ? query_role<NR>(a, w, sm, sh, lane)
               : several && a.n_heads % NR ? softmax_role<NR, true>(a, w, sm, sh, tmem, tm_s, parts, total, ctas, tid)
                                           : softmax_role<NR, false>(a, w, sm, sh, tmem, tm_s, parts, total, ctas, tid);
    };
    const bool ok = nr == 64   ? roles(std::integral_constant<int, 64>{})
                    : nr == 32 ? roles(std::integral_constant<int, 32>{})
                               : roles(std::integral_constant<int, 16>{});
    if (!ok)
        atomicOr(&g_paged_status, 1);
    pdl_launch_dependents();
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        tmem_free(tmem, kTmemCols);
    }
}

// Joins the parts of the split groups: a block takes one row of one group at
// a time, a thread four latent columns.  A group is named by the first CTA
// start that it crosses; every warp ranks the starts for itself, one lane a
// start, so that no barrier stands before the loads.  A warp's lanes hold the
// parts' (m, z), and the first parts' O are on their way while these are
// reduced.  Six blocks an SM, all resident at once: with twelve the second half
// starts over with the ranks (one request of 1531 tokens 14.8 us to 13.3).
constexpr int kJoinThreads = W8_LATENT_DIM / 4, kJoinBlocks = 6, kJoinDeep = 8, kMaxCtas = 1024;
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks)
    join_kernel(const __grid_constant__ w8_latent_paged a, void *ws, int ctas)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const Parts parts = parts_of(ws, ctas);
    pdl_wait();
    // the starts are taken 256 at a time: one pass on a GPU of up to 256 SMs
    constexpr int kStarts = 8, kSlot = kMaxRows * W8_LATENT_DIM / 4;
    int before = 0, job = blockIdx.x; // groups of the starts before c0
    for (int c0 = 0; c0 < ctas; c0 += 32 * kStarts) {
        int rank[kStarts], groups = before;
        bool yes[kStarts];
#pragma unroll
        for (int k = 0; k < kStarts; ++k) {
            const int c = c0 + 32 * k + lane;
            yes[k] = c >= 1 && c < ctas && parts.at[c].last >= 0;
        }
#pragma unroll
        for (int k = 0; k < kStarts; ++k) {
            const uint32_t all = __ballot_sync(0xffffffffu, yes[k]);
            rank[k] = yes[k] ? groups + __popc(all & ((1u << lane) - 1)) : -1;
            groups += __popc(all);
        }
        for (; job < groups * kMaxRows; job += gridDim.x) {
            const int row = job % kMaxRows;
            int at = 0;
#pragma unroll
            for (int k = 0; k < kStarts; ++k)
                at = rank[k] == job / kMaxRows ? c0 + 32 * k + lane : at;
            const Boundary b = parts.at[__reduce_max_sync(0xffffffffu, at)];
            if (row >= b.rows)
                continue;
            // part i lies in slot 2 (first + i), the first in the one after
            const int n = b.last - b.first + 1;
            const float2 *mz = parts.mz + 2 * b.first * kMaxRows + row;
            const float4 *from = reinterpret_cast<const float4 *>(parts.o) + size_t(2 * b.first) * kSlot + row * (W8_LATENT_DIM / 4) + tid;
            float m = -CUDART_INF_F, z = 0.0f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int i0 = 0; i0 < n; i0 += 32) {
                const int here = min(n - i0, 32);
                float2 part = make_float2(-CUDART_INF_F, 0.0f);
                if (lane < here)
                    part = mz[(2 * (i0 + lane) + (i0 + lane == 0)) * kMaxRows];
                float4 v[kJoinDeep];
                auto load = [&](int j) {
#pragma unroll
                    for (int i = 0; i < kJoinDeep; ++i)
                        if (j + i < here)
                            v[i] = from[size_t(2 * (i0 + j + i) + (i0 + j + i == 0)) * kSlot];
                };
                load(0);
                float top = part.x;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                top = fmaxf(top, m);
                const float ref = top == -CUDART_INF_F ? 0.0f : top;
                const float f0 = ex2(m - ref), e = ex2(part.x - ref); // 0 for a part that has seen nothing (its O is 0)
                m = top;
                float sum = part.y * e;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, d);
                z = fmaf(z, f0, sum);
                o.x *= f0;
                o.y *= f0;
                o.z *= f0;
                o.w *= f0;
#pragma unroll 1
                for (int j = 0; j < here; j += kJoinDeep) {
                    if (j > 0)
                        load(j);
#pragma unroll
                    for (int i = 0; i < kJoinDeep; ++i) {
                        const float f = __shfl_sync(0xffffffffu, e, j + i);
                        if (j + i < here) {
                            o.x = fmaf(v[i].x, f, o.x);
                            o.y = fmaf(v[i].y, f, o.y);
                            o.z = fmaf(v[i].z, f, o.z);
                            o.w = fmaf(v[i].w, f, o.w);
                        }
                    }
                }
            }
            const bool some = z > 0.0f || z != z;
            const float inv = some ? 1.0f / z : 0.0f;
            const int tok = (b.row0 + row) / a.n_heads, head = b.row0 + row - tok * a.n_heads;
            uint32_t *out = reinterpret_cast<uint32_t *>(a.out + tok * a.ld_out_tok + head * a.ld_out_head) + 2 * tid;
            out[0] = pack_bf16(o.x * inv, o.y * inv);
            out[1] = pack_bf16(o.z * inv, o.w * inv);
            if (a.lse && tid == 0)
                a.lse[b.row0 + row] = some ? (m + log2f(z)) * kLn2 : -CUDART_INF_F;
        }
        before = groups;
    }
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

} // namespace

bool encode_bf16_map(CUtensorMap *map, const void *base, int rank, const uint64_t *sizes, const uint64_t *strides,
                     const uint32_t *box)
{
    const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
    if (!enc)
        return false;
    cuuint64_t dims[3], str[2];
    cuuint32_t bx[3], one[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        dims[i] = sizes[i];
        bx[i] = box[i];
        if (i > 0)
            str[i - 1] = strides[i - 1];
    }
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void *>(base), dims, str, bx, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t latent_paged_ws_bytes(int, int, int, int sms) { return parts_bytes(sms); }

cudaError_t launch_latent_paged(const w8_latent_paged &a, void *ws, int sms, cudaStream_t s)
{
    if (sms > kMaxCtas)
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = raise_smem(raised, reinterpret_cast<const void *>(&paged_kernel), kSmem);
    if (e != cudaSuccess)
        return e;
    alignas(64) CUtensorMap map;
    const uint64_t sizes[3] = {W8_LATENT_ROW, uint64_t(a.cache.page_size), uint64_t(a.cache.n_pages)};
    const uint64_t strides[2] = {uint64_t(a.cache.ld_tok) * 2, uint64_t(a.cache.ld_page) * 2};
    const uint32_t box[3] = {64, uint32_t(a.cache.page_size < kTile ? a.cache.page_size : kTile), 1};
    if (!encode_bf16_map(&map, a.cache.data, 3, sizes, strides, box))
        return cudaErrorInvalidValue;
    e = launch_dependent(&paged_kernel, dim3(unsigned(sms)), kPagedThreads, kSmem, s, a, map, ws);
    if (e != cudaSuccess || sms < 2)
        return e;
    return launch_dependent(&join_kernel, dim3(unsigned(kJoinBlocks * sms)), kJoinThreads, 0, s, a, ws, sms);
}

cudaError_t paged_status(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_paged_status, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(int));
    }
    return e;
}

} // namespace w8
