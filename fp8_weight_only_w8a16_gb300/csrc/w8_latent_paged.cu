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
// Seven warps: 0-3 softmax (16 rows each; loads S, writes P as bf16 into shared
// memory, raises the reference, divides and stores), 4 copies (tensor-map
// boxes of min(page, 64) tokens x 64 columns), 5 and 6 issue the two products
// (a thread each: with one thread for both, a tile's second product waited
// for the next tile's copies, 4.8 us a tile instead of XXX).  The ring
// frees latent columns in units of 128 as the second product passes over
// them; the rope chunk has a ring of its own and is free after the first.
// The reference moves only when a row's maximum passes it by 2^8 (p stays
// below 2^8, and 2^8 of fp32's range costs no precision): O is then rescaled
// in tensor memory, for most inputs once or twice in the first tiles.
//
// The work is cut by tiles, not by requests: all groups' tiles in one line,
// an equal run a CTA, one CTA an SM.  A group that more than one run touches
// leaves its parts (O, m, z in fp32) in the workspace, and a second kernel
// joins them.  Lengths are read on the device; the line's length picks NR:
// 64 rows a group, or fewer when there are not enough tiles to give every SM
// one.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "w8_device.cuh"
#include "w8_serve_internal.h"
#include "w8_tcgen.cuh"

namespace w8 {

__device__ int g_paged_status;

namespace {

using namespace tcg;

constexpr int kTile = 64;                    // tokens
constexpr int kChunk = kTile * 128;          // bytes of 64 tokens x 64 columns
constexpr int kUnit = 2 * kChunk;            // 128 latent columns
constexpr int kMaxRows = 64;
constexpr int kPagedThreads = 224, kSoftThreads = 128, kCopyWarp = 4, kScoreWarp = 5, kOutWarp = 6;
constexpr int kMaxUnits = 12, kMaxRopes = 3;
constexpr int kSmem = 227 * 1024 - 2048;     // what the CTA takes; the rest is static
constexpr int kTmemCols = 512;
constexpr float kRaise = 8.0f;               // log2 of how far a row's weights may pass 1
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Shared memory for groups of nr rows: Q, P, then the rings.
struct Smem {
    int q, p, rope, unit, ropes, units;
};
__host__ __device__ constexpr Smem smem_plan(int nr)
{
    Smem s{};
    s.q = 0;
    s.p = s.q + 9 * nr * 128;
    s.rope = s.p + nr * 128;
    s.ropes = nr == 64 ? 2 : 3;
    s.unit = s.rope + s.ropes * kChunk;
    s.units = (kSmem - 1024 - s.unit) / kUnit;
    s.units = s.units > kMaxUnits ? kMaxUnits : s.units;
    return s;
}
static_assert(smem_plan(64).units >= 8 && smem_plan(32).units >= 8 && smem_plan(16).units >= 8, "two tiles in flight");
// the first product reads 64 rows from every chunk of Q: the last chunk's
// reach past Q stays inside the allocation
static_assert(smem_plan(16).unit >= 8 * 16 * 128 + kChunk, "Q's reach");

// What the parts of split groups need: [2 CTAs][64][512] fp32, [2 CTAs][64]
// (m, z), [CTAs] the group that runs over the CTA's start.
struct Boundary {
    int first, last; // CTAs that hold the group's parts; last < 0: none starts before this CTA
    int row0, rows;  // the group's rows, counted over all query tokens' heads
    int first_slot;  // the first CTA's part
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
// Tiles of group g: those its last row sees, one (of nothing) if that is none.
__device__ __forceinline__ int group_tiles(const Request &q, int heads, int nr, int g)
{
    const int last = min((g + 1) * nr, q.q * heads) - 1;
    const int n = (seen(q, last / heads) + kTile - 1) / kTile;
    return n < 1 ? 1 : n;
}
__device__ __forceinline__ int groups_of(const Request &q, int heads, int nr) { return (q.q * heads + nr - 1) / nr; }

// One CTA's place in the line of tiles, a run of one group at a time.  Every
// role walks it for itself.
struct Walk {
    int64_t pos, end;  // the next tile, the CTA's last + 1
    int r, g, off;     // its request, group, place in the group
    Request req;
    int tiles;         // of the group
    int run;           // tiles of this run

    __device__ __forceinline__ bool next(const w8_latent_paged &a, int nr, bool first)
    {
        if (!first) {
            pos += run;
            off = 0;
            if (pos < end && ++g >= groups_of(req, a.n_heads, nr)) {
                g = 0;
                do
                    req = request_of(a, ++r);
                while (req.q == 0 && r + 1 < a.n_req);
            }
        } else if (pos < end) {
            req = request_of(a, r);
        }
        if (pos >= end)
            return false;
        tiles = group_tiles(req, a.n_heads, nr, g);
        run = int(min(int64_t(tiles - off), end - pos));
        return true;
    }
};

// 2 KB at most: the rest is the rings'.
struct Shared {
    uint64_t unit_full[kMaxUnits], unit_free[kMaxUnits];
    uint64_t rope_full[kMaxRopes], rope_free[kMaxRopes];
    uint64_t q, s[2], s_free[2], p, o, end[2];
    int64_t out[kMaxRows]; // a row's place in the output
    int64_t sum[kPagedThreads / 32];
    int max[kPagedThreads / 32];
    int start[3];
    uint32_t tmem;
    float f[kMaxRows], inv[kMaxRows];
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

// One lane of a converged warp.  Tensor-core steps issued by a lane that the
// compiler only knows as `lane == 0` take 85 to 130 cycles each whatever their
// shape; issued under this they take their own 32 to 128.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Keys that the last row of the walk's group sees.
__device__ __forceinline__ int group_sees(const w8_latent_paged &a, const Walk &w, int nr)
{
    return seen(w.req, (min((w.g + 1) * nr, w.req.q * a.n_heads) - 1) / a.n_heads);
}

// ---- copies ---------------------------------------------------------------
template <int NR>
__device__ __forceinline__ bool copy_role(const w8_latent_paged &a, const CUtensorMap &map, Walk w, uint8_t *sm, Shared &sh,
                                          int lane)
{
    constexpr Smem lay = smem_plan(NR);
    // lane l of a unit's copies: chunk l / boxes, box l % boxes
    const int page = a.cache.page_size, box = min(page, kTile), boxes = kTile / box;
    const int shift = 31 - __clz(page), bx = lane % boxes, c = lane / boxes;
    Turn un, rn;
    int units = 0, ropes = 0; // copied so far
    bool ok = true;
    for (bool first = true; ok && w.next(a, NR, first); first = false) {
        const int32_t *table = a.block_table + int64_t(w.r) * a.ld_table;
        const int vis = group_sees(a, w, NR);
        // this lane's page of a tile; the next tile's is fetched ahead
        auto page_of = [&](int t) {
            const int j = t * kTile + bx * box;
            int pg = a.cache.n_pages; // reads as zeros
            if (t < w.off + w.run && j < vis) {
                pg = __ldg(table + (j >> shift));
                pg = pg < 0 || pg > a.cache.n_pages ? a.cache.n_pages : pg;
            }
            return pg;
        };
        int pg = page_of(w.off);
        for (int t = w.off; ok && t < w.off + w.run; ++t) {
            const int j0 = t * kTile, left = min(vis - j0, kTile);
            if (left <= 0)
                break;
            const int need = (left + box - 1) / box; // boxes with a key that is seen
            const int y = (j0 + bx * box) & (page - 1);
            const int ahead = page_of(t + 1);
            for (int u = 0; u < 5; ++u) {
                const bool rope = u == 4;
                const int k = rope ? rn.k : un.k;
                uint64_t *full = rope ? &sh.rope_full[k] : &sh.unit_full[k];
                if (rope ? ropes >= lay.ropes : units >= lay.units)
                    ok = __all_sync(0xffffffffu, rope ? bar_wait(&sh.rope_free[k], rn.parity ^ 1)
                                                      : bar_wait(&sh.unit_free[k], un.parity ^ 1));
                if (!ok)
                    break;
                const int chunks = rope ? 1 : 2;
                if (lane == 0)
                    bar_expect(full, uint32_t(chunks * need * box * 128));
                __syncwarp();
                if (c < chunks && bx < need)
                    copy_box(smem_addr(sm + (rope ? lay.rope + k * kChunk : lay.unit + k * kUnit) + c * kChunk + bx * box * 128),
                             &map, 64 * (2 * u + c), y, pg, full);
                if (rope) {
                    rn.step(lay.ropes);
                    ++ropes;
                } else {
                    un.step(lay.units);
                    ++units;
                }
            }
            pg = ahead;
        }
    }
    // the copies still in flight (there are any only after a wait elsewhere gave up)
    for (int i = max(0, units - lay.units); i < units; ++i)
        bar_wait(&sh.unit_full[i % lay.units], uint32_t((i / lay.units) & 1));
    for (int i = max(0, ropes - lay.ropes); i < ropes; ++i)
        bar_wait(&sh.rope_full[i % lay.ropes], uint32_t((i / lay.ropes) & 1));
    return ok;
}

// ---- first product ----------------------------------------------------------
template <int NR>
__device__ __forceinline__ bool score_role(const w8_latent_paged &a, Walk w, uint8_t *sm, Shared &sh, uint32_t tm_s)
{
    constexpr Smem lay = smem_plan(NR);
    constexpr uint32_t id = inst_desc(64, kTile, false, false);
    const uint64_t dq = desc128_k(smem_addr(sm + lay.q), 1024);
    const uint64_t drope = desc128_k(smem_addr(sm + lay.rope), 1024), dunit = desc128_k(smem_addr(sm + lay.unit), 1024);
    const bool one = elect_one();
    Turn un, rn;
    int runs = 0, n = 0; // runs with keys, tiles
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) { ok = __all_sync(0xffffffffu, ok && bar_wait(bar, parity & 1)); };
    for (bool first = true; ok && w.next(a, NR, first); first = false) {
        if (group_sees(a, w, NR) == 0)
            continue;
        wait(&sh.q, uint32_t(runs));
        ++runs;
        for (int t = 0; ok && t < w.run; ++t, ++n) {
            // S of tile n - 2, in the same columns, has been read
            if (n >= 2)
                wait(&sh.s_free[n & 1], uint32_t(n / 2 - 1));
            const uint32_t d = tm_s + uint32_t(n & 1) * kTile;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                wait(&sh.unit_full[un.k], un.parity);
                if (!ok)
                    break;
                fence_after();
                const uint64_t dk = dunit + uint64_t((un.k * kUnit) >> 4);
                if (one) {
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_ss(d, dq + uint64_t(((2 * u + s / 4) * NR * 128 + (s % 4) * 32) >> 4),
                               dk + uint64_t(((s / 4) * kChunk + (s % 4) * 32) >> 4), id, uint32_t(u | s));
                }
                __syncwarp();
                un.step(lay.units);
            }
            wait(&sh.rope_full[rn.k], rn.parity);
            if (!ok)
                break;
            fence_after();
            const uint64_t dk = drope + uint64_t((rn.k * kChunk) >> 4);
            if (one) {
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma_ss(d, dq + uint64_t((8 * NR * 128 + s * 32) >> 4), dk + uint64_t((s * 32) >> 4), id, 1);
                commit(&sh.rope_free[rn.k]);
                commit(&sh.s[n & 1]);
            }
            __syncwarp();
            rn.step(lay.ropes);
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
    const uint64_t dp = desc128_k(smem_addr(sm + lay.p), 1024), dunit = desc128(smem_addr(sm + lay.unit), kChunk, 1024);
    const bool one = elect_one();
    Turn un;
    int n = 0;
    bool ok = true;
    for (bool first = true; ok && w.next(a, NR, first); first = false) {
        if (group_sees(a, w, NR) == 0)
            continue;
        for (int t = 0; ok && t < w.run; ++t, ++n) {
            ok = __all_sync(0xffffffffu, bar_wait(&sh.p, uint32_t(n & 1)));
            if (!ok)
                break;
            fence_after();
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint64_t dv = dunit + uint64_t((un.k * kUnit) >> 4);
                if (one) {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        mma_ss(tmem + uint32_t(u * NR), dv + uint64_t((s * 2048) >> 4), dp + uint64_t((s * 32) >> 4), id,
                               uint32_t(t | s));
                    commit(&sh.unit_free[un.k]);
                }
                __syncwarp();
                un.step(lay.units);
            }
            if (one)
                commit(&sh.o);
            __syncwarp();
        }
    }
    if (one)
        commit(&sh.end[1]);
    __syncwarp();
    return bar_wait(&sh.end[1], 0) && ok;
}

// ---- softmax, output --------------------------------------------------------
template <int NR>
__device__ __forceinline__ bool softmax_role(const w8_latent_paged &a, Walk w, uint8_t *sm, Shared &sh, uint32_t tmem,
                                             uint32_t tm_s, const Parts &parts, int64_t total, int64_t ctas, int tid)
{
    constexpr Smem lay = smem_plan(NR);
    const int warp = tid >> 5, lane = tid & 31;
    const float sl = a.scale * kLog2e;
    const int g4 = lane >> 2, t4 = lane & 3;
    const bool active = 16 * warp < NR; // warps that have rows
    const uint32_t lanes = uint32_t(32 * warp) << 16;
    bool ok = true;
    // a wait that gave up is followed by no other, but every barrier below is
    // still met, so that no warp waits for one that left
    auto wait = [&](uint64_t *bar, int phase) { ok = __all_sync(0xffffffffu, ok && bar_wait(bar, uint32_t(phase & 1))); };
    if (tid == 0 && (w.pos >= w.end || w.off == 0))
        parts.at[blockIdx.x].last = -1; // no group runs over this CTA's start
    // the rows' places in Q, while Q is loaded, where P will be
    int64_t *const q_at = reinterpret_cast<int64_t *>(sm + lay.p);
    int n = 0; // tiles so far
    for (bool first = true; w.next(a, NR, first); first = false) {
        const int row0 = w.g * NR, rows = min(NR, w.req.q * a.n_heads - row0);
        const int vis = seen(w.req, (row0 + rows - 1) / a.n_heads);
        // the two rows of this thread: how many keys they see
        int lim[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 16 * warp + g4 + 8 * h;
            lim[h] = row < rows ? seen(w.req, (row0 + row) / a.n_heads) : 0;
        }
        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, z[2] = {0.0f, 0.0f};
        if (tid < rows) {
            const int tok = w.req.q0 + (row0 + tid) / a.n_heads, head = (row0 + tid) % a.n_heads;
            sh.out[tid] = tok * a.ld_out_tok + head * a.ld_out_head;
            q_at[tid] = tok * a.ld_qlat_tok + head * a.ld_qlat_head;
            q_at[NR + tid] = tok * a.ld_qrope_tok + head * a.ld_qrope_head;
        }
        sync_some(1, kSoftThreads);
        if (vis > 0) {
            // Q: 72 vectors of 16 bytes a row, nine loads of a thread in flight
            constexpr int kBatch = 9;
#pragma unroll 1
            for (int i0 = 0; i0 < NR * 72; i0 += kBatch * kSoftThreads) {
                uint4 x[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int i = i0 + b * kSoftThreads + tid, row = i / 72, v = i - row * 72;
                    x[b] = make_uint4(0, 0, 0, 0);
                    if (row < rows)
                        x[b] = __ldg(reinterpret_cast<const uint4 *>(v < 64 ? a.q_lat + q_at[row] + 8 * v
                                                                            : a.q_rope + q_at[NR + row] + 8 * (v - 64)));
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int i = i0 + b * kSoftThreads + tid, row = i / 72, v = i - row * 72;
                    *reinterpret_cast<uint4 *>(sm + lay.q + (v >> 3) * NR * 128 + row * 128 + (((v & 7) ^ (row & 7)) << 4)) =
                        x[b];
                }
            }
            fence_async_shared();
            bar_arrive(&sh.q);
            for (int t = 0; t < w.run; ++t, ++n) {
                const int j0 = (w.off + t) * kTile;
                wait(&sh.s[n & 1], n >> 1);
                fence_after();
                float f[2] = {1.0f, 1.0f};
                float x[32];
                bool raise = false;
                if (active) {
                    ld16x64(x, tm_s + lanes + uint32_t(n & 1) * kTile);
                    wait_ld();
                }
                fence_before();
                bar_arrive(&sh.s_free[n & 1]);
                if (active) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (j0 + kTile > lim[h]) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (j0 + 8 * (i >> 1) + 2 * t4 + (i & 1) >= lim[h])
                                    x[4 * (i >> 1) + 2 * h + (i & 1)] = -CUDART_INF_F;
                        }
                        float mx = x[2 * h];
#pragma unroll
                        for (int i = 1; i < 16; ++i)
                            mx = fmaxf(mx, x[4 * (i >> 1) + 2 * h + (i & 1)]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        mx *= sl;
                        if (m[h] == -CUDART_INF_F) {
                            m[h] = mx; // nothing summed yet
                        } else if (mx > m[h] + kRaise) {
                            f[h] = ex2(m[h] - mx);
                            m[h] = mx;
                            z[h] *= f[h];
                            raise = true;
                        }
                        const float ref = m[h] == -CUDART_INF_F ? 0.0f : m[h];
                        float sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float &e = x[4 * (i >> 1) + 2 * h + (i & 1)];
                            e = ex2(fmaf(e, sl, -ref));
                            sum += e;
                        }
                        z[h] += sum;
                    }
                }
                // the last tile's second product has read P and written O
                if (t > 0)
                    wait(&sh.o, n - 1);
                if (active) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = 16 * warp + g4 + 8 * h;
                        uint8_t *p = sm + lay.p + row * 128 + 4 * t4;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint32_t *>(p + ((j ^ (row & 7)) << 4)) =
                                pack_bf16(x[4 * j + 2 * h], x[4 * j + 2 * h + 1]);
                        if (t4 == 0)
                            sh.f[row] = f[h];
                    }
                }
                if (j0 + kTile > vis) {
                    // rows of the tile that nobody sees may hold anything: their weights are 0, 0 x NaN is not
                    const int dead = kTile - (vis - j0);
                    for (int i = tid; i < dead * 64; i += kSoftThreads) {
                        const int c = i / (dead * 8), rest = i - c * dead * 8;
                        const int k = (4 * n + c / 2) % lay.units;
                        *reinterpret_cast<uint4 *>(sm + lay.unit + k * kUnit + (c & 1) * kChunk + (vis - j0) * 128 +
                                                   rest * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                if (sync_any(1, kSoftThreads, raise)) {
                    fence_after();
#pragma unroll 1
                    for (int c = 0; c < NR / 4; ++c) { // 16 columns: rows 16 c % NR .. of block 16 c / NR
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
                fence_before();
                fence_async_shared();
                bar_arrive(&sh.p);
            }
            wait(&sh.o, n - 1);
            fence_after();
        }
        // ---- the run's result: the output, or a part of it
        const bool whole = w.off == 0 && w.run == w.tiles;
        const int slot = 2 * int(blockIdx.x) + (w.off == 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            z[h] += __shfl_xor_sync(0xffffffffu, z[h], 1);
            z[h] += __shfl_xor_sync(0xffffffffu, z[h], 2);
            const int row = 16 * warp + g4 + 8 * h;
            if (active && t4 == 0) {
                const bool some = z[h] > 0.0f || z[h] != z[h];
                sh.inv[row] = some ? 1.0f / z[h] : 0.0f;
                if (row < rows) {
                    if (!whole)
                        parts.mz[slot * kMaxRows + row] = make_float2(m[h], z[h]);
                    else if (a.lse)
                        a.lse[int64_t(w.req.q0) * a.n_heads + row0 + row] =
                            some ? (m[h] + log2f(z[h])) * kLn2 : -CUDART_INF_F;
                }
            }
        }
        if (w.off > 0 && tid == 0) {
            // the group runs over this CTA's start
            const int64_t s0 = w.pos - w.off, s1 = s0 + w.tiles - 1; // the group's tiles in the line
            Boundary b;
            b.first = int(((s0 + 1) * ctas - 1) / total);
            b.last = int(((s1 + 1) * ctas - 1) / total);
            b.row0 = w.req.q0 * a.n_heads + row0;
            b.rows = rows;
            b.first_slot = 2 * b.first + 1;
            parts.at[blockIdx.x] = b;
        }
        sync_some(1, kSoftThreads);
#pragma unroll 1
        for (int c = 0; c < NR / 4; ++c) {
            const int n0 = (16 * c) % NR, d0 = 128 * (16 * c / NR) + 32 * warp;
            if (n0 >= rows)
                continue;
            float o[16];
            if (vis > 0) {
                ld32x16(o, tmem + lanes + uint32_t(16 * c));
                wait_ld();
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[i] = 0.0f;
            }
            if (whole) {
                // lane pairs trade halves, so that each stores two columns of one row
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float e = o[i] * sh.inv[n0 + i], d = o[i + 1] * sh.inv[n0 + i + 1];
                    const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? e : d, 1);
                    const int row = n0 + i + (lane & 1);
                    if (row < rows)
                        *reinterpret_cast<uint32_t *>(a.out + sh.out[row] + d0 + (lane & ~1)) =
                            lane & 1 ? pack_bf16(got, d) : pack_bf16(e, got);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (n0 + i < rows)
                        parts.o[(size_t(slot) * kMaxRows + n0 + i) * W8_LATENT_DIM + d0 + lane] = o[i];
            }
        }
        fence_before(); // the loads of O, before the next run's products
        sync_some(1, kSoftThreads); // the rows' places and 1 / z are read
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
        for (int i = 0; i < kMaxUnits; ++i) {
            bar_init(&sh.unit_full[i], 1);
            bar_init(&sh.unit_free[i], 1);
        }
        for (int i = 0; i < kMaxRopes; ++i) {
            bar_init(&sh.rope_full[i], 1);
            bar_init(&sh.rope_free[i], 1);
        }
        bar_init(&sh.q, kSoftThreads);
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

    // ---- the line of tiles: its length, NR, this CTA's run -------------------
    const int per = (a.n_req + kPagedThreads - 1) / kPagedThreads;
    const int r0 = min(tid * per, a.n_req), r1 = min(r0 + per, a.n_req);
    int nr = kMaxRows;
    int64_t mine = 0, before = 0, total = 0;
    for (;;) {
        mine = 0;
        int rows = 0;
        for (int r = r0; r < r1; ++r) {
            const Request q = request_of(a, r);
            rows = max(rows, min(q.q * a.n_heads, kMaxRows));
            const int n = groups_of(q, a.n_heads, nr);
            for (int g = 0; g < n; ++g)
                mine += group_tiles(q, a.n_heads, nr, g);
        }
        int64_t inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
            inc += lane >= d ? o : 0;
            rows = max(rows, __shfl_xor_sync(0xffffffffu, rows, d));
        }
        __syncthreads(); // the last pass's sums are read
        if (lane == 31) {
            sh.sum[warp] = inc;
            sh.max[warp] = rows;
        }
        __syncthreads();
        before = inc - mine;
        total = 0;
        rows = 0;
        for (int w = 0; w < kPagedThreads / 32; ++w) {
            before += w < warp ? sh.sum[w] : 0;
            total += sh.sum[w];
            rows = max(rows, sh.max[w]);
        }
        // fewer rows a group: when no group would be filled, or when that
        // many more groups still leave no SM two tiles
        const int half = nr / 2;
        if (nr == 16 || !(rows <= half || total * 2 <= gridDim.x))
            break;
        nr = half;
    }
    const int64_t ctas = min(total, int64_t(gridDim.x)); // those that have work
    Walk w{};
    w.pos = ctas ? min(int64_t(blockIdx.x), ctas) * total / ctas : 0;
    w.end = ctas ? min(int64_t(blockIdx.x) + 1, ctas) * total / ctas : 0;
    if (w.pos < w.end && before <= w.pos && w.pos < before + mine) {
        int64_t at = before;
        for (int r = r0; r < r1; ++r) {
            const Request q = request_of(a, r);
            const int n = groups_of(q, a.n_heads, nr);
            for (int g = 0; g < n; ++g) {
                const int t = group_tiles(q, a.n_heads, nr, g);
                if (at <= w.pos && w.pos < at + t) {
                    sh.start[0] = r;
                    sh.start[1] = g;
                    sh.start[2] = int(w.pos - at);
                }
                at += t;
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem, tm_s = tmem + 4 * kMaxRows; // O in columns 0 .., S after it
    w.r = sh.start[0];
    w.g = sh.start[1];
    w.off = sh.start[2];
    const Parts parts = parts_of(ws, int(gridDim.x));
    const int role = __shfl_sync(0xffffffffu, warp, 0);
    auto roles = [&](auto rows) {
        constexpr int NR = decltype(rows)::value;
        return role == kCopyWarp    ? copy_role<NR>(a, map, w, sm, sh, lane)
               : role == kScoreWarp ? score_role<NR>(a, w, sm, sh, tm_s)
               : role == kOutWarp   ? out_role<NR>(a, w, sm, sh, tmem)
                                    : softmax_role<NR>(a, w, sm, sh, tmem, tm_s, parts, total, ctas, tid);
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

// Joins the parts of a split group: a block a (CTA start, row), a thread four
// latent columns.  The block of the group's first crossed start does it.
__global__ void __launch_bounds__(W8_LATENT_DIM / 4)
    join_kernel(const __grid_constant__ w8_latent_paged a, void *ws, int ctas)
{
    __shared__ float s_w[1024];
    __shared__ float s_m[4], s_z[4];
    const int tid = threadIdx.x, cta = blockIdx.x + 1, row = blockIdx.y;
    pdl_wait();
    const Parts parts = parts_of(ws, ctas);
    const Boundary b = parts.at[cta];
    if (b.last < 0 || b.first != cta - 1 || row >= b.rows)
        return;
    const int n = b.last - b.first + 1;
    // part i: the first CTA's, then slot 2 c of each later one
    auto slot = [&](int i) { return size_t(i ? 2 * (b.first + i) : b.first_slot) * kMaxRows + row; };
    // the weights 2^(m_i - m): one pass for m, one for the sum
    float m = -CUDART_INF_F;
    for (int i = tid; i < n; i += blockDim.x)
        m = fmaxf(m, parts.mz[slot(i)].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((tid & 31) == 0)
        s_m[tid >> 5] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    const float ref = m == -CUDART_INF_F ? 0.0f : m;
    float z = 0.0f;
    for (int i = tid; i < n; i += blockDim.x) {
        const float2 mz = parts.mz[slot(i)];
        const float f = mz.x == -CUDART_INF_F ? 0.0f : ex2(mz.x - ref); // nothing seen: O is 0
        s_w[i] = f;
        z += mz.y * f;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        z += __shfl_xor_sync(0xffffffffu, z, d);
    if ((tid & 31) == 0)
        s_z[tid >> 5] = z;
    __syncthreads();
    z = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
        const float4 v = reinterpret_cast<const float4 *>(parts.o + slot(i) * W8_LATENT_DIM)[tid];
        const float f = s_w[i];
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
    }
    const bool some = z > 0.0f || z != z;
    const float inv = some ? 1.0f / z : 0.0f;
    const int tok = (b.row0 + row) / a.n_heads, head = (b.row0 + row) % a.n_heads;
    uint32_t *out = reinterpret_cast<uint32_t *>(a.out + tok * a.ld_out_tok + head * a.ld_out_head) + 2 * tid;
    out[0] = pack_bf16(o.x * inv, o.y * inv);
    out[1] = pack_bf16(o.z * inv, o.w * inv);
    if (a.lse && tid == 0)
        a.lse[b.row0 + row] = some ? (m + log2f(z)) * kLn2 : -CUDART_INF_F;
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
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(&paged_kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
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
    const int64_t rows = int64_t(a.n_tok) * a.n_heads;
    return launch_dependent(&join_kernel, dim3(unsigned(sms - 1), unsigned(rows < kMaxRows ? rows : kMaxRows)),
                            W8_LATENT_DIM / 4, 0, s, a, ws, sms);
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
