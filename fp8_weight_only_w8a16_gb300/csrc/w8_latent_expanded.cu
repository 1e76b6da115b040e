// w8_latent_expanded.cu -- latent attention, expanded form, over the keys and
// values of a prompt (w8_latent_attn_expanded).
//
// The kernel for few queries (mathematics and softmax: w8_expanded.cuh; many
// take pairs of CTAs, w8_latent_pair.cu).  A CTA takes 128 queries of one head.
// Both products run on tcgen05 with fp32 accumulators in tensor memory:
//   S [128 x 128] = Q K^T  (16 or 12 steps of 64 cycles)
//   O [128 x d_v] += P V   (8 steps of 128 or 64 cycles), P as bf16 in tensor
//     memory, in the columns of the S that it was made from.
// S has two buffers, so that the scores of the next tile are made while the
// weights of this one are.  With d_v = 256 the 512 columns are full: O 256,
// S 2 x 128.
//
// Ten warps: 0-7 softmax (two threads a row, 64 keys each), 8 copies, 9
// tensor-core issue.  Keys and values come by tensor-map copies into a ring of
// equal slots, in the order in which the steps use them: K of tile 0, then K
// of tile i + 1 and V of tile i in turn.  A K slot holds 128 keys x 64 or 128
// columns, K-major; a V slot 64 keys x d_v columns, MN-major.  The parts of a
// head's key (its own columns, the rope columns all heads share) meet only in
// shared memory.
//
// Measured (replayed): three prompts of 37 to 611 tokens at 16 heads of 128 + 64
// / 128 in 11.9 us, bound by the chain scores - softmax - output of a tile; a
// full tile of 192 + 64 / 256 takes 2566 cycles, 2048 of them steps, and wants
// 50 bytes a cycle and SM from L2.
#include "w8_copies.h"
#include "w8_expanded.cuh"

namespace w8 {

__device__ int g_expanded_status;

namespace {

using namespace expanded;

template <int DN, int DV>
struct Shape {
    static constexpr int kCols = DN + W8_LATENT_ROPE;      // of a query and a key
    static constexpr int kChunks = kCols / 64;
    static constexpr int kSlot = DV / 64 * 64 * 128;       // bytes
    static constexpr int kKChunks = kSlot / (kKeys * 128); // 64-column chunks of a K slot
    static constexpr int kKSlots = kChunks / kKChunks, kVSlots = kKeys / 64; // of a tile
    static constexpr int kQ = kChunks * kRows * 128;
    static constexpr int kSlots = (kSmem - 1024 - kQ) / kSlot;
    static constexpr int kS = DV; // S's first column; O starts at 0
    static_assert(kKSlots * kKChunks == kChunks && kS + 2 * kKeys <= kTmemCols && kSlots >= 4, "plan");
};
constexpr int kMaxSlots = 12;

struct Shared {
    uint64_t full[kMaxSlots], free_[kMaxSlots];
    uint64_t q, s[2], p[2], o, end;
    int count[kExpThreads / 32];
    int found[6];
    uint32_t tmem;
    float top[4][2][32];
};
static_assert(sizeof(Shared) <= 2048, "shared memory");

// What a CTA works on.
struct Item {
    int q0, rows;   // first query token, queries (of the CTA)
    int k0, nk;     // first key, keys of the request
    int see0;       // keys that the first query sees, uncut; one more for each later one (causal)
    int tiles;      // key tiles; 0: nothing is seen
};

template <int DN, int DV>
__global__ void __launch_bounds__(kExpThreads, 1)
    expanded_kernel(const __grid_constant__ w8_latent_expanded a, const __grid_constant__ Maps maps, int tiles_max)
{
    using S = Shape<DN, DV>;
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ __align__(16) Shared sh;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    uint8_t *const sm = s_dyn + ((1024u - (smem_addr(s_dyn) & 1023u)) & 1023u);
    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            bar_init(&sh.full[i], 1);
            bar_init(&sh.free_[i], 1);
        }
        bar_init(&sh.q, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.s[i], 1);
            bar_init(&sh.p[i], 32 * kSoftWarps);
        }
        bar_init(&sh.o, 1);
        bar_init(&sh.end, 1);
        bar_init_fence();
        sh.found[0] = -1;
    }
    if (warp == 0)
        tmem_alloc(&sh.tmem, kTmemCols);
    pdl_wait();

    // ---- the item: query tile `want` of all requests' tiles, last ones first ----
    const int head = int(blockIdx.x) / tiles_max;
    const int want = tiles_max - 1 - (int(blockIdx.x) - head * tiles_max);
    {
        const int per = (a.n_req + kExpThreads - 1) / kExpThreads;
        const int r0 = min(tid * per, a.n_req), r1 = min(r0 + per, a.n_req);
        auto queries = [&](int r, int &q0) {
            q0 = min(max(__ldg(a.cu_q + r), 0), a.n_q);
            return min(max(__ldg(a.cu_q + r + 1), q0), a.n_q) - q0;
        };
        int mine = 0, q0;
        for (int r = r0; r < r1; ++r)
            mine += (queries(r, q0) + kRows - 1) / kRows;
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            inc += lane >= d ? o : 0;
        }
        if (lane == 31)
            sh.count[warp] = inc;
        __syncthreads();
        int at = inc - mine;
        for (int i = 0; i < warp; ++i)
            at += sh.count[i];
        for (int r = r0; r < r1; ++r) {
            const int nq = queries(r, q0), n = (nq + kRows - 1) / kRows;
            if (at <= want && want < at + n) {
                const int k0 = min(max(__ldg(a.cu_k + r), 0), a.n_k);
                const int nk = min(max(__ldg(a.cu_k + r + 1), k0), a.n_k) - k0;
                const int i0 = (want - at) * kRows;
                sh.found[0] = q0 + i0;
                sh.found[1] = min(kRows, nq - i0);
                sh.found[2] = k0;
                sh.found[3] = nk;
                sh.found[4] = a.causal ? nk - nq + i0 + 1 : nk;
            }
            at += n;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem, tm_s = tmem + S::kS;
    Item it;
    it.q0 = sh.found[0];
    it.rows = sh.found[1];
    it.k0 = sh.found[2];
    it.nk = sh.found[3];
    it.see0 = sh.found[4];
    // keys that row i sees
    auto sees = [&](int i) { return min(max(it.see0 + (a.causal ? i : 0), 0), it.nk); };
    it.tiles = it.q0 < 0 ? 0 : (sees(it.rows - 1) + kKeys - 1) / kKeys;

    bool ok = true;
    if (it.q0 < 0) {
        // fewer tiles than the grid allows for
    } else if (warp == kCopyWarp) {
        if (it.tiles > 0 && elect_one()) {
            const uint32_t ring = smem_addr(sm + S::kQ), q = smem_addr(sm);
            bar_expect(&sh.q, S::kQ);
#pragma unroll
            for (int c = 0; c < S::kChunks; ++c)
                copy_box(q + c * kRows * 128, c < DN / 64 ? &maps.q_nope : &maps.q_rope, c < DN / 64 ? 64 * c : 0, head, it.q0,
                         &sh.q, policy_normal());
            Ring<S::kSlots> to;
            auto slot = [&]() { // the next slot, its old content read
                ok = ok && to.take([&](int k, uint32_t parity) { return bar_wait(&sh.free_[k], parity); });
                return ok;
            };
            for (int i = 0; i <= it.tiles && ok; ++i) {
                if (i < it.tiles) {
#pragma unroll
                    for (int g = 0; g < S::kKSlots; ++g) {
                        if (!slot())
                            break;
                        bar_expect(&sh.full[to.k], S::kSlot);
#pragma unroll
                        for (int c = 0; c < S::kKChunks; ++c) {
                            const int chunk = g * S::kKChunks + c;
                            const uint32_t dst = ring + uint32_t(to.k * S::kSlot + c * kKeys * 128);
                            if (chunk < DN / 64)
                                copy_box(dst, &maps.k_nope, 64 * chunk, head, it.k0 + i * kKeys, &sh.full[to.k], policy_normal());
                            else
                                copy_box(dst, &maps.k_rope, 0, it.k0 + i * kKeys, &sh.full[to.k]);
                        }
                        to.filled();
                    }
                }
                if (i > 0) {
#pragma unroll
                    for (int g = 0; g < S::kVSlots; ++g) {
                        if (!slot())
                            break;
                        bar_expect(&sh.full[to.k], S::kSlot);
#pragma unroll
                        for (int c = 0; c < DV / 64; ++c)
                            copy_box(ring + uint32_t(to.k * S::kSlot + c * 64 * 128), &maps.v, 64 * c, head,
                                     it.k0 + (i - 1) * kKeys + 64 * g, &sh.full[to.k], policy_normal());
                        to.filled();
                    }
                }
            }
            // The copies still in flight.  (Not only where a wait of this lane gave up:
            // the lanes that use them may have.)
            bar_wait(&sh.q, 0);
            to.drain([&](int k, uint32_t parity) { bar_wait(&sh.full[k], parity); });
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (it.tiles > 0) {
            constexpr uint32_t id_s = inst_desc(kRows, kKeys, false, false), id_o = inst_desc(kRows, DV, false, true);
            const uint64_t dq = desc128_k(smem_addr(sm), 1024), dk = desc128_k(smem_addr(sm + S::kQ), 1024),
                           dv = desc128(smem_addr(sm + S::kQ), 64 * 128, 1024);
            const bool one = elect_one();
            int k = 0;
            uint32_t parity = 0;
            auto wait = [&](uint64_t *bar, uint32_t ph) { ok = __all_sync(0xffffffffu, ok && bar_wait(bar, ph & 1)); };
            auto step = [&] {
                if (++k == S::kSlots) {
                    k = 0;
                    parity ^= 1;
                }
            };
            wait(&sh.q, 0);
            for (int i = 0; i <= it.tiles && ok; ++i) {
                if (i < it.tiles) {
                    // the second product of tile i - 2 has read its weights, in the same columns
                    if (i >= 2)
                        wait(&sh.o, uint32_t(i - 2));
                    const uint32_t d = tm_s + uint32_t(i & 1) * kKeys;
#pragma unroll
                    for (int g = 0; g < S::kKSlots; ++g) {
                        wait(&sh.full[k], parity);
                        fence_after();
                        const uint64_t b = dk + uint64_t((k * S::kSlot) >> 4);
                        if (one && ok) {
#pragma unroll
                            for (int c = 0; c < 4 * S::kKChunks; ++c)
                                mma_ss(d, dq + uint64_t((g * S::kKChunks * kRows * 128 + (c / 4) * kRows * 128 + (c % 4) * 32) >> 4),
                                       b + uint64_t(((c / 4) * kKeys * 128 + (c % 4) * 32) >> 4), id_s, uint32_t(g | c));
                            commit(&sh.free_[k]);
                        }
                        __syncwarp();
                        step();
                    }
                    if (one)
                        commit(&sh.s[i & 1]);
                    __syncwarp();
                }
                if (i > 0) {
                    const int t = i - 1;
                    wait(&sh.p[t & 1], uint32_t(t >> 1));
                    const uint32_t p = tm_s + uint32_t(t & 1) * kKeys;
#pragma unroll
                    for (int g = 0; g < S::kVSlots; ++g) {
                        wait(&sh.full[k], parity);
                        fence_after();
                        const uint64_t b = dv + uint64_t((k * S::kSlot) >> 4);
                        if (one && ok) {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                mma_ts(tmem, p + uint32_t(64 * g + 8 * c), b + uint64_t((c * 2048) >> 4), id_o, uint32_t(t | g | c));
                            commit(&sh.free_[k]);
                        }
                        __syncwarp();
                        step();
                    }
                    if (one)
                        commit(&sh.o);
                    __syncwarp();
                }
            }
            // nothing is in the tensor cores when the CTA frees its memory
            if (one)
                commit(&sh.end);
            __syncwarp();
            ok = bar_wait(&sh.end, 0) && ok;
        }
    } else {
        // ---- softmax, output: thread (row, half) ------------------------------------
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
        const float sl = a.scale * kLog2e;
        const uint32_t lanes = uint32_t(32 * quarter) << 16;
        const int lim = row < it.rows ? sees(row) : 0;
        auto wait = [&](uint64_t *bar, int ph) { ok = __all_sync(0xffffffffu, ok && bar_wait(bar, uint32_t(ph & 1))); };
        float m = -CUDART_INF_F, z = 0.0f;
        for (int t = 0; t < it.tiles; ++t) {
            wait(&sh.s[t & 1], t >> 1);
            fence_after();
            softmax_half<DV>(tm_s + lanes + uint32_t((t & 1) * kKeys + 64 * half), tmem + lanes, t * kKeys + 64 * half, lim, sl,
                             t == 0, quarter, half, lane, sh.top[quarter], m, z, [&] { wait(&sh.o, t - 1); });
            if (t == it.tiles - 1 && it.nk < it.tiles * kKeys) {
                // values past the request's keys may be anything: their weights are 0, 0 x NaN is not
                const int first = it.nk - t * kKeys, slot0 = it.tiles * S::kKSlots + t * S::kVSlots;
                for (int g = first / 64; g < S::kVSlots; ++g) {
                    const int k = (slot0 + g) % S::kSlots;
                    wait(&sh.full[k], (slot0 + g) / S::kSlots);
                    const int from = max(first - 64 * g, 0), n = (64 - from) * 8; // 16-byte vectors of a run
                    for (int i = tid; i < n * (DV / 64); i += 32 * kSoftWarps)
                        *reinterpret_cast<uint4 *>(sm + S::kQ + k * S::kSlot + i / n * 64 * 128 + from * 128 + i % n * 16) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_async_shared();
            }
            // (waited for before this tile's output can be made, so that the
            // barrier is never two uses ahead of a warp)
            if (t > 0)
                wait(&sh.o, t - 1);
            fence_before();
            bar_arrive(&sh.p[t & 1]);
        }
        if (it.tiles > 0)
            wait(&sh.o, it.tiles - 1);
        fence_after();
        sh.top[quarter][half][lane] = z;
        sync_some(1 + quarter, 64);
        z = sh.top[quarter][0][lane] + sh.top[quarter][1][lane];
        const bool some = z > 0.0f || z != z;
        const float inv = some ? 1.0f / z : 0.0f;
        if (row < it.rows && half == 0 && a.lse)
            a.lse[(int64_t(it.q0) + row) * a.n_heads + head] = some ? (m + log2f(z)) * kLn2 : -CUDART_INF_F;
        // The rows go out through shared memory, where Q was (every score is
        // made), so that a warp stores whole rows: a lane's row straight from
        // tensor memory took 32 half-used sectors a store, 4 us a CTA.
        uint8_t *const stage = sm + 32 * quarter * DV * 2; // of this pair of warps
        float zero = 0.0f;
#pragma unroll
        for (int c = 0; c < DV / 2; c += 32)
            stage32(stage, DV * 2, tmem + lanes + uint32_t(DV / 2 * half + c), it.tiles > 0, inv, (DV / 2 * half + c) / 8, lane, zero);
        sync_some(1 + quarter, 64);
        constexpr int kVecs = DV / 8, kAtOnce = 32 / kVecs; // vectors of a row, rows of a store
#pragma unroll 4
        for (int r = 16 * half; r < 16 * half + 16; r += kAtOnce) {
            const int mine = r + lane / kVecs, v = lane % kVecs, i = 32 * quarter + mine;
            if (i < it.rows)
                *reinterpret_cast<uint4 *>(a.out + (int64_t(it.q0) + i) * a.ld_out_tok + head * a.ld_out_head + 8 * v) =
                    *reinterpret_cast<const uint4 *>(stage + mine * DV * 2 + ((v ^ (mine & 7)) << 4));
        }
        if (a.causal) {
            const bool bad = zero != zero && z - z == 0.0f && row < it.rows && lim < it.nk;
            if (sync_any(1 + quarter, 64, bad)) // the rows are stored
                redo_rows<DN, DV>(a, __ballot_sync(0xffffffffu, bad), it.q0 + 32 * quarter, head, it.k0, min(it.tiles * kKeys, it.nk), lim,
                                  m, z, half, lane);
        }
    }
    if (!ok)
        atomicOr(&g_expanded_status, 1);
    pdl_launch_dependents();
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        tmem_free(tmem, kTmemCols);
    }
}

template <int DN, int DV>
cudaError_t launch(const w8_latent_expanded &a, cudaStream_t s)
{
    auto *fn = &expanded_kernel<DN, DV>;
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = raise_smem(raised, reinterpret_cast<const void *>(fn), kSmem);
    if (e != cudaSuccess)
        return e;
    Maps maps;
    if (!map_all(maps, a, kKeys, 64))
        return cudaErrorInvalidValue;
    // query tiles: every request may end in a part of one
    const int64_t tiles = a.n_q / kRows + (a.n_req < a.n_q ? a.n_req : a.n_q);
    if (tiles * a.n_heads > INT32_MAX)
        return cudaErrorInvalidValue;
    return launch_dependent(fn, dim3(unsigned(tiles * a.n_heads)), kExpThreads, kSmem, s, a, maps, int(tiles));
}

} // namespace

cudaError_t launch_latent_expanded(const w8_latent_expanded &a, int sms, cudaStream_t s)
{
    // Pairs of CTAs halve what comes from L2 and run on from item to item, but
    // start later and pad queries to 256: they pay from about five waves of
    // 128-query tiles on, of requests that fill their tiles.  64 heads of
    // 192 + 64 / 256, one prompt of 4096: 367 us in pairs, 387 by CTAs; of 2048:
    // 123 and 128; of 1024: 50.9 and 50.4; 32 requests of 20: 136 and 113; 16
    // heads, 9 requests of 700: 65 and 70; one of 1024: 26 and 16.  (64 heads of
    // 128 + 64 / 128, one prompt of 4096: 304 and 296.)
    if (int64_t(a.n_q) * a.n_heads >= int64_t(5) * kRows * sms && a.n_q / a.n_req >= 512)
        return launch_expanded_pairs(a, s);
    return a.d_nope == 192 ? launch<192, 256>(a, s) : launch<128, 128>(a, s);
}

cudaError_t expanded_status(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_expanded_status, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_expanded_status, &zero, sizeof(int));
    }
    return e;
}

} // namespace w8
