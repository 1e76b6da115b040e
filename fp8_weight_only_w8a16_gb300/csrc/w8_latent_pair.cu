// w8_latent_pair.cu -- latent attention, expanded form, for prompts that fill
// the GPU: pairs of CTAs (mathematics and softmax: w8_expanded.cuh).
//
// A pair (a cluster of two SMs) takes 256 queries of one head.  Both products
// run on tcgen05 over the pair (cta_group::2), each CTA's 128 rows in its own
// tensor memory:
//   S [256 x 128] = Q K^T  (16 or 12 steps of 64 cycles)
//   O [256 x d_v] += P V   (8 steps of 128 or 64 cycles), P as bf16 in tensor
//     memory, in the columns of the S that it was made from.
// Each CTA copies half of a tile -- 64 of its keys, d_v / 2 of its value columns
// -- and the tensor cores of both read both halves.  A CTA with whole tiles for
// itself needs 64 bytes a cycle and SM from L2 at full rate and gets about 50.
// S has two buffers, so that the scores of the next tile are made while the
// weights of this one are.  With d_v = 256 the 512 columns are full: O 256,
// S 2 x 128.
//
// Ten warps a CTA: 0-7 softmax and output (two threads a row, 64 keys each), 8
// copies, 9 tensor-core issue (the pair's first CTA only).  Keys and values come by tensor-map copies
// into a ring of slots, in the order in which the steps use them: K of tile 0,
// then K of tile i + 1 and V of tile i in turn.  A K slot holds 64 keys, K-major,
// a V slot 128 keys x d_v / 2 columns, MN-major.  Slots fill on a barrier of the
// first CTA, which counts both halves' bytes; steps that are done arrive in both.
//
// The grid has a pair for every (head, query tile), the longest first within a
// head, heads one after the other (152 SMs then work on about five heads, whose
// keys stay in L2).  A resident pair, once it has its item, takes the next one
// off the grid by cancelling a launch (clusterlaunchcontrol), so that the next
// item's copies and first scores run while this one's output is stored.
//
// Measured (replayed): a prompt of 4096 at 64 heads of 192 + 64 / 256 in 366 to
// 384 us by the clock, 1.5 PFLOP/s at best, tensor pipe 64 %.  A tile takes 2310 cycles of which 2048
// are steps: the scores of tile i + 2 wait for the output of tile i, whose
// weights lie in the same columns, and nothing else is left to run meanwhile.
// The rest is the 3400 cycles of an item's output, of which the next one's
// scores hide about half, and the clock (the chip is at its power limit).
#include <stddef.h>

#include "w8_copies.h"
#include "w8_expanded.cuh"

namespace w8 {

__device__ int g_pairs_status;

namespace {

using namespace expanded;

constexpr int kPairRows = 2 * kRows;
constexpr int kMaxSlots = 8;

template <int DN, int DV>
struct Shape {
    static constexpr int kCols = DN + W8_LATENT_ROPE;      // of a query and a key
    static constexpr int kChunks = kCols / 64;
    static constexpr int kHalf = kKeys / 2 * 128;          // bytes of 64 columns of a CTA's keys
    static constexpr int kK = kChunks * kHalf;             // of a CTA's half of a tile's keys
    static constexpr int kRuns = DV / 128;                 // 64-column runs of a CTA's half of the values
    static constexpr int kRun = kKeys * 128;
    static constexpr int kV = kRuns * kRun;
    static constexpr int kSlot = kK > kV ? kK : kV;
    static constexpr int kQ = kChunks * kRows * 128;
    static constexpr int kStage = kRows * 256;             // output on its way: 128 columns of every row
    static constexpr int kFit = (kSmem - 1024 - kQ - kStage) / kSlot;
    static constexpr int kSlots = kFit < kMaxSlots ? kFit : kMaxSlots;
    static constexpr int kS = DV; // S's first column; O starts at 0
    static_assert(kSlot % 1024 == 0 && kS + 2 * kKeys <= kTmemCols && kSlots >= 4, "plan");
};

struct Shared {
    uint64_t full[kMaxSlots], free_[kMaxSlots], v_last[kMaxSlots];
    uint64_t q, q_free, s[2], p[2], o, done, end;
    uint64_t next_full[2], next_free[2];
    uint4 next[2];               // answers of the grid
    int before[kExpThreads];     // query tiles up to each thread's run of requests, inclusive
    int count[kExpThreads / 32];
    uint32_t tmem;
    int failed;                  // a wait of either CTA gave up
    PairIssued issued[2];        // by this CTA, by the other
};
static_assert(sizeof(Shared) <= 2048, "shared memory");

// What a pair works on, as one of its CTAs sees it.
struct Item {
    int q0, rows;   // first query token, queries (of the CTA; 0 or fewer: none)
    int k0, nk;     // first key, keys of the request
    int see0;       // keys that the CTA's first row sees, uncut; one more for each later one (causal)
    int tiles;      // key tiles of the pair; 0: nothing is seen; -1: no such item
    int head;
};

// The same place in a CTA of the pair, in its first.
__device__ __forceinline__ uint32_t in_cta(const void *p, int rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t in_first(const void *p) { return in_cta(p, 0); }
__device__ __forceinline__ void pair_store(uint32_t to, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
}
// Arrive at a barrier of either CTA.  What passes between the two CTAs this way
// lies in tensor memory and in the async proxy's view of shared memory, completed
// by tcgen05.wait and proxy fences before; no value in ordinary memory does, so
// the arrival carries no wider release (one of cluster scope took 1000 cycles).
__device__ __forceinline__ void pair_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pair_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Box copies into this CTA whose bytes count on a barrier of either CTA.
__device__ __forceinline__ void pair_copy(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
                 "{%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void pair_copy(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
                 "{%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
// Steps over the pair: A rows 0 .. 127 in the first CTA, 128 .. 255 in the
// second, each half of B in its CTA.
__device__ __forceinline__ void pair_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// Arrive on this barrier of both CTAs once every step issued so far is done.
__device__ __forceinline__ void pair_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_addr(bar)),
                 "h"(uint16_t(3))
                 : "memory");
}
// Ask for a pair that has not been launched yet; both CTAs get the answer at the
// same place, 16 bytes on the same barrier.
__device__ __forceinline__ void ask_next(uint4 *answer, uint64_t *bar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 "
                 "[%0], [%1];" ::"r"(smem_addr(answer)),
                 "r"(smem_addr(bar))
                 : "memory");
}
// Its number; -1 if there is none left.
__device__ __forceinline__ int answered(const uint4 *answer)
{
    uint32_t some, x;
    asm volatile("{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%2];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
                 : "=r"(some), "=r"(x)
                 : "r"(smem_addr(answer))
                 : "memory");
    return some ? int(x >> 1) : -1;
}

// The barriers of a CTA, as pair_drain sees them.
template <typename S>
struct DrainBars {
    Shared &sh;
    __device__ __forceinline__ void forgo(uint64_t *bar, uint32_t bytes)
    {
        asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
    }
    __device__ __forceinline__ void wait_last(int s, uint32_t parity) { bar_wait(&sh.v_last[s], parity); }
    __device__ __forceinline__ void wait_full(int s, uint32_t parity) { bar_wait(&sh.full[s], parity); }
    __device__ __forceinline__ void expect_full(int s, bool values) { bar_expect(&sh.full[s], values ? S::kV : S::kK); }
    __device__ __forceinline__ void forgo_full(int s, bool values) { forgo(&sh.full[s], values ? S::kV : S::kK); }
    __device__ __forceinline__ void wait_queries(uint32_t parity) { bar_wait(&sh.q, parity); }
    __device__ __forceinline__ void expect_queries() { bar_expect(&sh.q, S::kQ); }
    __device__ __forceinline__ void forgo_queries() { forgo(&sh.q, S::kQ); }
    __device__ __forceinline__ void wait_answer(int k, uint32_t parity) { bar_wait(&sh.next_full[k], parity); }
    __device__ __forceinline__ void expect_answer(int k) { bar_expect(&sh.next_full[k], 16); }
};

__device__ __forceinline__ int queries(const w8_latent_expanded &a, int r, int &q0)
{
    q0 = min(max(__ldg(a.cu_q + r), 0), a.n_q);
    return min(max(__ldg(a.cu_q + r + 1), q0), a.n_q) - q0;
}

// The item of pair `id`; a whole warp asks.
__device__ __forceinline__ Item find(const w8_latent_expanded &a, const Shared &sh, int id, int tiles_max, int rank, int lane)
{
    Item it;
    it.head = id / tiles_max;
    it.tiles = -1;
    it.q0 = it.rows = it.k0 = it.nk = it.see0 = 0;
    const int want = tiles_max - 1 - (id - it.head * tiles_max); // last ones first
    // the run of requests that holds it, then the request
    int run = 0;
#pragma unroll
    for (int i = 0; i < kExpThreads; i += 32)
        run += __popc(__ballot_sync(0xffffffffu, sh.before[i + lane] <= want));
    if (run == kExpThreads)
        return it; // fewer tiles than the grid allows for
    const int per = (a.n_req + kExpThreads - 1) / kExpThreads, end = min((run + 1) * per, a.n_req);
    int at = run ? sh.before[run - 1] : 0;
    for (int r0 = run * per; r0 < end; r0 += 32) {
        int q0 = 0, nq = 0;
        if (r0 + lane < end)
            nq = queries(a, r0 + lane, q0);
        const int n = (nq + kPairRows - 1) / kPairRows;
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            inc += lane >= d ? o : 0;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, at + inc > want);
        if (here) {
            const int src = __ffs(int(here)) - 1, r = r0 + src;
            const int i0 = (want - at - __shfl_sync(0xffffffffu, inc - n, src)) * kPairRows;
            nq = __shfl_sync(0xffffffffu, nq, src);
            q0 = __shfl_sync(0xffffffffu, q0, src);
            it.k0 = min(max(__ldg(a.cu_k + r), 0), a.n_k);
            it.nk = min(max(__ldg(a.cu_k + r + 1), it.k0), a.n_k) - it.k0;
            const int last = min(i0 + kPairRows, nq) - 1;
            it.tiles = (min(max(a.causal ? it.nk - nq + last + 1 : it.nk, 0), it.nk) + kKeys - 1) / kKeys;
            it.q0 = q0 + i0 + rank * kRows;
            it.rows = min(nq - i0 - rank * kRows, kRows);
            it.see0 = a.causal ? it.nk - nq + i0 + rank * kRows + 1 : it.nk;
            return it;
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
    }
    return it;
}

template <int DN, int DV>
__global__ void __launch_bounds__(kExpThreads, 1)
    pair_kernel(const __grid_constant__ w8_latent_expanded a, const __grid_constant__ Maps maps, int tiles_max)
{
    using S = Shape<DN, DV>;
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ __align__(16) Shared sh;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = int(blockIdx.x & 1); // the cluster is two CTAs along x
    uint8_t *const sm = s_dyn + ((1024u - (smem_addr(s_dyn) & 1023u)) & 1023u);
    uint8_t *const s_stage = sm + S::kQ, *const s_ring = s_stage + S::kStage;
    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            bar_init(&sh.full[i], 1);
            bar_init(&sh.free_[i], 1);
            bar_init(&sh.v_last[i], 1);
        }
        bar_init(&sh.q, 1);
        bar_init(&sh.q_free, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.s[i], 1);
            bar_init(&sh.p[i], 2 * kSoftWarps);
            bar_init(&sh.next_full[i], 1);
            bar_init(&sh.next_free[i], 2 * (kSoftWarps + 1) + 1);
        }
        bar_init(&sh.o, 1);
        bar_init(&sh.done, 2 * kSoftWarps);
        bar_init(&sh.end, 1);
        bar_init_fence();
        sh.failed = 0;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    // ---- query tiles up to each thread's run of requests -----------------------
    {
        const int per = (a.n_req + kExpThreads - 1) / kExpThreads;
        const int r0 = min(tid * per, a.n_req), r1 = min(r0 + per, a.n_req);
        int mine = 0, q0;
        for (int r = r0; r < r1; ++r)
            mine += (queries(a, r, q0) + kPairRows - 1) / kPairRows;
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            inc += lane >= d ? o : 0;
        }
        if (lane == 31)
            sh.count[warp] = inc;
        __syncthreads();
        for (int i = 0; i < warp; ++i)
            inc += sh.count[i];
        sh.before[tid] = inc;
    }
    fence_before();
    __syncthreads();
    pair_sync(); // both CTAs' barriers are ready, and both have their tensor memory
    fence_after();
    const uint32_t tmem = sh.tmem, tm_s = tmem + S::kS;

    // Every role runs over the pair's items: its own pair's, then what the grid
    // answers.  next() is asked once an item, by whole warps.
    bool ok = true;
    int id = int(blockIdx.x >> 1), items = 0;
    const uint32_t next_free0 = in_first(&sh.next_free[0]);
    auto next = [&] { // into id
        const int k = items & 1;
        ok = __all_sync(0xffffffffu, ok && bar_wait(&sh.next_full[k], uint32_t((items >> 1) & 1)));
        id = ok ? answered(&sh.next[k]) : -1;
        fence_async_shared(); // read before the next answer is written there
        __syncwarp();
        if (lane == 0)
            pair_arrive(next_free0 + uint32_t(8 * k));
        ++items;
    };

    if (warp == kCopyWarp) {
        Ring<S::kSlots> to;
        PairIssued did{};
        int work = 0; // items with keys
        const uint32_t ring = smem_addr(s_ring), q = smem_addr(sm), q_bar = in_first(&sh.q);
        while (id >= 0) {
            // the answer for the item after this one
            const int n = items & 1;
            if (items >= 2 && rank == 0)
                ok = __all_sync(0xffffffffu, ok && bar_wait(&sh.next_free[n], uint32_t(((items >> 1) - 1) & 1)));
            if (elect_one()) {
                bar_expect(&sh.next_full[n], 16);
                if (rank == 0 && ok)
                    ask_next(&sh.next[n], &sh.next_full[n]);
            }
            ++did.expects;
            did.asks += rank == 0 && ok;
            __syncwarp();
            const Item it = find(a, sh, id, tiles_max, rank, lane);
            if (it.tiles > 0) {
                uint32_t who;
                if (elect_one(who)) {
                    auto slot = [&]() { // the next slot, its old content read
                        ok = ok && to.take([&](int k, uint32_t parity) { return bar_wait(&sh.free_[k], parity); });
                        return ok;
                    };
                    if (work > 0)
                        ok = ok && bar_wait(&sh.q_free, uint32_t((work - 1) & 1));
                    if (ok) {
                        // (rows past the request's queries are another's, or past the tensor and zero: their results are dropped)
                        if (rank == 0)
                            bar_expect(&sh.q, 2 * S::kQ);
#pragma unroll
                        for (int c = 0; c < S::kChunks; ++c)
                            pair_copy(q + c * kRows * 128, c < DN / 64 ? &maps.q_nope : &maps.q_rope, c < DN / 64 ? 64 * c : 0,
                                      it.head, it.q0, q_bar);
                        ++did.queries;
                    }
                    for (int i = 0; i <= it.tiles; ++i) {
                        if (i < it.tiles) {
                            if (!slot())
                                break;
                            const uint32_t bar = in_first(&sh.full[to.k]), dst = ring + uint32_t(to.k * S::kSlot);
                            if (rank == 0)
                                bar_expect(&sh.full[to.k], 2 * S::kK);
                            const int row = it.k0 + i * kKeys + rank * (kKeys / 2);
#pragma unroll
                            for (int c = 0; c < S::kChunks; ++c) {
                                if (c < DN / 64)
                                    pair_copy(dst + c * S::kHalf, &maps.k_nope, 64 * c, it.head, row, bar);
                                else
                                    pair_copy(dst + c * S::kHalf, &maps.k_rope, 0, row, bar);
                            }
                            did.full ^= 1u << to.k;
                            did.values &= ~(1u << to.k);
                            to.filled();
                        }
                        if (i > 0) {
                            if (!slot())
                                break;
                            // the last tile's values count here: their rows past the keys are made zero before they are used
                            const bool last = i == it.tiles;
                            const uint32_t bar = last ? smem_addr(&sh.v_last[to.k]) : in_first(&sh.full[to.k]);
                            if (last)
                                bar_expect(&sh.v_last[to.k], S::kV);
                            else if (rank == 0)
                                bar_expect(&sh.full[to.k], 2 * S::kV);
#pragma unroll
                            for (int c = 0; c < S::kRuns; ++c)
                                pair_copy(ring + uint32_t(to.k * S::kSlot + c * S::kRun), &maps.v, rank * (DV / 2) + 64 * c, it.head,
                                          it.k0 + (i - 1) * kKeys, bar);
                            if (last) {
                                did.last ^= 1u << to.k;
                            } else {
                                did.full ^= 1u << to.k;
                                did.values |= 1u << to.k;
                            }
                            to.filled();
                        }
                    }
                }
                __syncwarp();
                ok = __shfl_sync(0xffffffffu, ok, who);
                to.k = __shfl_sync(0xffffffffu, to.k, who);
                to.used = __shfl_sync(0xffffffffu, to.used, who);
                to.parity = __shfl_sync(0xffffffffu, to.parity, who);
                did.full = __shfl_sync(0xffffffffu, did.full, who);
                did.values = __shfl_sync(0xffffffffu, did.values, who);
                did.last = __shfl_sync(0xffffffffu, did.last, who);
                did.queries = __shfl_sync(0xffffffffu, did.queries, who);
                ++work;
            }
            next();
        }
        // what has been issued, for either CTA's last waits
        did.used = uint32_t(to.used);
        if (lane == 0) {
            // The products' last arrivals come to both CTAs, and only the first, which
            // issues them, waits for its own: the second may not leave before they are here.
            if (rank == 1 && ok) {
                auto wait = [&](uint64_t *bar, uint32_t parity) { ok = ok && bar_wait(bar, parity); };
                to.drain([&](int k, uint32_t parity) { wait(&sh.free_[k], parity); });
                wait(&sh.q_free, (did.queries & 1u) ^ 1u); // (none copied: the phase before the first, ended)
                wait(&sh.end, 0);
            }
            sh.issued[0] = did;
            const uint32_t there = in_cta(&sh.issued[1], rank ^ 1);
            pair_store(there + offsetof(PairIssued, full), did.full);
            pair_store(there + offsetof(PairIssued, values), did.values);
            pair_store(there + offsetof(PairIssued, last), did.last);
            pair_store(there + offsetof(PairIssued, used), did.used);
            pair_store(there + offsetof(PairIssued, queries), did.queries);
            pair_store(there + offsetof(PairIssued, expects), did.expects);
            pair_store(there + offsetof(PairIssued, asks), did.asks);
        }
    } else if (warp == kMmaWarp && rank == 0) {
        constexpr uint32_t id_s = inst_desc(kPairRows, kKeys, false, false), id_o = inst_desc(kPairRows, DV, false, true);
        const uint64_t dq = desc128_k(smem_addr(sm), 1024), dk = desc128_k(smem_addr(s_ring), 1024),
                       dv = desc128(smem_addr(s_ring), S::kRun, 1024);
        int k = 0, work = 0, n = 0; // slot, items with keys, tiles of the items before
        uint32_t parity = 0;        // of `full`, a bit a slot (an item's last values do not use it)
        for (Item it = find(a, sh, id, tiles_max, rank, lane); id >= 0;) {
            // A step of the item: the scores of tile i, then the output of tile
            // i - 1.  The next item is asked for before the last of them, while
            // the softmax of the last tile runs.
            auto steps = [&](int i0, int i1) {
                uint32_t who;
                if (elect_one(who)) {
                    auto wait = [&](uint64_t *bar, int ph) { ok = ok && bar_wait(bar, uint32_t(ph & 1)); };
                    auto filled = [&] {
                        wait(&sh.full[k], int(parity >> k & 1));
                        parity ^= 1u << k;
                    };
                    auto step = [&] { k = k + 1 == S::kSlots ? 0 : k + 1; };
                    if (i0 == 0)
                        wait(&sh.q, work);
                    for (int i = i0; i < i1; ++i) {
                        if (i < it.tiles) {
                            const int t = n + i;
                            filled();
                            // The second product of tile t - 2 has read its weights, in
                            // the same columns.  (Every use of the barrier is waited for
                            // before the next but one can come: an item's last product
                            // waits for the one before it.)
                            if (i > 0 && t >= 2)
                                wait(&sh.o, t - 2);
                            if (!ok)
                                break;
                            fence_after();
                            const uint32_t d = tm_s + uint32_t(t & 1) * kKeys;
                            const uint64_t b = dk + uint64_t((k * S::kSlot) >> 4);
#pragma unroll
                            for (int c = 0; c < 4 * S::kChunks; ++c)
                                pair_mma_ss(d, dq + uint64_t(((c / 4) * kRows * 128 + (c % 4) * 32) >> 4),
                                            b + uint64_t(((c / 4) * S::kHalf + (c % 4) * 32) >> 4), id_s, uint32_t(c));
                            pair_commit(&sh.s[t & 1]);
                            pair_commit(&sh.free_[k]);
                            if (i == it.tiles - 1)
                                pair_commit(&sh.q_free);
                            step();
                        }
                        if (i > 0) {
                            const int t = n + i - 1;
                            if (i < it.tiles)
                                filled();
                            else if (t > 0)
                                wait(&sh.o, t - 1);
                            if (i == 1 && work > 0) // the last item's output has been read
                                wait(&sh.done, work - 1);
                            wait(&sh.p[t & 1], t >> 1);
                            if (!ok)
                                break;
                            fence_after();
                            const uint32_t p = tm_s + uint32_t(t & 1) * kKeys;
                            const uint64_t b = dv + uint64_t((k * S::kSlot) >> 4);
#pragma unroll
                            for (int c = 0; c < kKeys / 16; ++c)
                                pair_mma_ts(tmem, p + uint32_t(64 * (c / 4) + 8 * (c % 4)), b + uint64_t((c * 2048) >> 4), id_o,
                                            uint32_t((i - 1) | c));
                            pair_commit(&sh.o);
                            pair_commit(&sh.free_[k]);
                            step();
                        }
                    }
                }
                __syncwarp();
                ok = __shfl_sync(0xffffffffu, ok, who);
                k = __shfl_sync(0xffffffffu, k, who);
                parity = __shfl_sync(0xffffffffu, parity, who);
            };
            if (it.tiles > 0)
                steps(0, it.tiles);
            next();
            Item then = it;
            if (id >= 0)
                then = find(a, sh, id, tiles_max, rank, lane);
            if (it.tiles > 0) {
                const bool more = ok;
                ok = true; // a failed wait for the answer does not keep the output back
                steps(it.tiles, it.tiles + 1);
                ok = ok && more;
                n += it.tiles;
                ++work;
            }
            it = then;
        }
        // nothing is in the tensor cores when the CTAs free their memory
        if (elect_one())
            pair_commit(&sh.end);
        __syncwarp();
        ok = bar_wait(&sh.end, 0) && ok;
    } else if (warp == kMmaWarp) {
        // the first CTA's issues for both
    } else {
        // ---- softmax, output: thread (row, half) ------------------------------------
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
        const float sl = a.scale * kLog2e;
        const uint32_t o_at = tmem + (uint32_t(32 * quarter) << 16), s_at = o_at + S::kS;
        uint8_t *const stage = s_stage + quarter * 32 * 256; // of this pair of warps
        float(*const top)[32] = reinterpret_cast<float(*)[32]>(stage);
        auto wait = [&](uint64_t *bar, int ph) { ok = __all_sync(0xffffffffu, ok && bar_wait(bar, uint32_t(ph & 1))); };
        const uint32_t p_bar = in_first(&sh.p[0]), done_bar = in_first(&sh.done);
        int n = 0, slots = 0; // tiles, slots of the items before
        uint32_t last_parity = 0; // of v_last, a bit a slot
        for (Item it = find(a, sh, id, tiles_max, rank, lane); id >= 0;) {
            // keys that this thread's row sees
            const int lim = row < it.rows ? min(max(it.see0 + (a.causal ? row : 0), 0), it.nk) : 0;
            float m = -CUDART_INF_F, z = 0.0f;
            Item then = it;
            auto look_ahead = [&] { // the next item, found while the tensor cores are at the last tile
                next();
                if (id >= 0)
                    then = find(a, sh, id, tiles_max, rank, lane);
            };
            for (int t = 0; t < it.tiles; ++t, ++n) {
                if (t == it.tiles - 1)
                    look_ahead();
                wait(&sh.s[n & 1], n >> 1);
                fence_after();
                softmax_half<DV>(s_at + uint32_t((n & 1) * kKeys + 64 * half), o_at, t * kKeys + 64 * half, lim, sl, t == 0, quarter,
                                 half, lane, top, m, z, [&] { wait(&sh.o, n - 1); });
                if (t == it.tiles - 1) {
                    // this CTA's half of the last values is here; rows past the
                    // request's keys may be anything: their weights are 0, 0 x NaN is not
                    const int k = (slots + 2 * it.tiles - 1) % S::kSlots;
                    wait(&sh.v_last[k], int(last_parity >> k & 1));
                    last_parity ^= 1u << k;
                    const int from = it.nk - t * kKeys;
                    if (from < kKeys) {
                        uint8_t *v = s_ring + k * S::kSlot;
                        const int vecs = (kKeys - from) * 8; // 16-byte vectors of a run
                        for (int i = tid; i < vecs * S::kRuns; i += 32 * kSoftWarps)
                            *reinterpret_cast<uint4 *>(v + i / vecs * S::kRun + from * 128 + i % vecs * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_async_shared();
                }
                // (waited for before this tile's output can be made, so that the
                // barrier is never two uses ahead of a warp)
                if (n > 0)
                    wait(&sh.o, n - 1);
                fence_before();
                __syncwarp();
                if (lane == 0)
                    pair_arrive(p_bar + uint32_t(8 * (n & 1)));
            }
            if (it.tiles <= 0)
                look_ahead();
            float zero = 0.0f;
            if (it.tiles >= 0) {
                if (it.tiles > 0)
                    wait(&sh.o, n - 1);
                fence_after();
                top[half][lane] = z;
                sync_some(1 + quarter, 64);
                z = top[0][lane] + top[1][lane];
                sync_some(1 + quarter, 64);
                const bool some = z > 0.0f || z != z;
                const float inv = some ? 1.0f / z : 0.0f;
                if (row < it.rows && half == 0 && a.lse)
                    a.lse[(int64_t(it.q0) + row) * a.n_heads + it.head] = some ? (m + log2f(z)) * kLn2 : -CUDART_INF_F;
                // The rows go out through shared memory, 128 columns at a time, so
                // that a warp stores runs of 256 bytes (a lane's row straight from
                // tensor memory took 32 half-used sectors a store).
#pragma unroll
                for (int c = 0; c < DV; c += 128) {
                    if (c > 0)
                        sync_some(1 + quarter, 64); // the columns before are stored
#pragma unroll
                    for (int e = 0; e < 64; e += 32)
                        stage32(stage, 256, o_at + uint32_t(c + 64 * half + e), it.tiles > 0, inv, 8 * half + e / 8, lane, zero);
                    if (c + 128 == DV && it.tiles > 0) { // O is read
                        fence_before();
                        __syncwarp();
                        if (lane == 0)
                            pair_arrive(done_bar);
                    }
                    sync_some(1 + quarter, 64);
#pragma unroll
                    for (int r = 16 * half; r < 16 * half + 16; r += 2) {
                        const int mine = r + lane / 16, v = lane % 16, i = 32 * quarter + mine;
                        if (i < it.rows)
                            *reinterpret_cast<uint4 *>(a.out + (int64_t(it.q0) + i) * a.ld_out_tok + it.head * a.ld_out_head + c +
                                                       8 * v) =
                                *reinterpret_cast<const uint4 *>(stage + mine * 256 + ((v ^ (mine & 7)) << 4));
                    }
                }
            }
            slots += 2 * max(it.tiles, 0);
            // The rows are stored before `top` is written again; and the two warps
            // leave together when either has given up.
            if (sync_any(1 + quarter, 64, !ok)) {
                ok = false;
                break;
            }
            if (a.causal) {
                const uint32_t bad = __ballot_sync(0xffffffffu, zero != zero && z - z == 0.0f && row < it.rows && lim < it.nk);
                if (bad)
                    redo_rows<DN, DV>(a, bad, it.q0 + 32 * quarter, it.head, it.k0, min(it.tiles * kKeys, it.nk), lim, m, z, half, lane);
            }
            it = then;
        }
    }
    if (!ok) {
        atomicOr(&g_pairs_status, 1);
        sh.failed = 1;
        pair_store(in_cta(&sh.failed, rank ^ 1), 1);
    }
    pdl_launch_dependents();
    fence_before();
    __syncthreads();
    pair_sync(); // neither CTA leaves while the other's steps or arrivals may reach it
    if (sh.failed) { // in both CTAs or in neither: copies may be on their way, to phases that nobody has waited for
        if (warp == kCopyWarp && lane == 0) {
            DrainBars<S> bars{sh};
            pair_drain(sh.issued[0], sh.issued[1], rank == 0, S::kSlots, bars);
        }
        __syncthreads();
        pair_sync();
    }
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int DN, int DV>
cudaError_t launch(const w8_latent_expanded &a, cudaStream_t s)
{
    auto *fn = &pair_kernel<DN, DV>;
    static std::atomic<uint64_t> raised{0};
    const cudaError_t e = raise_smem(raised, reinterpret_cast<const void *>(fn), kSmem);
    if (e != cudaSuccess)
        return e;
    Maps maps;
    if (!map_all(maps, a, kKeys / 2, kKeys))
        return cudaErrorInvalidValue;
    // query tiles: every request may end in a part of one
    const int64_t tiles = a.n_q / kPairRows + (a.n_req < a.n_q ? a.n_req : a.n_q);
    if (2 * tiles * a.n_heads > INT32_MAX)
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(2 * tiles * a.n_heads));
    cfg.blockDim = dim3(kExpThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, a, maps, int(tiles));
}

} // namespace

cudaError_t launch_expanded_pairs(const w8_latent_expanded &a, cudaStream_t s)
{
    return a.d_nope == 192 ? launch<192, 256>(a, s) : launch<128, 128>(a, s);
}

cudaError_t pairs_status(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_pairs_status, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_pairs_status, &zero, sizeof(int));
    }
    return e;
}

} // namespace w8
