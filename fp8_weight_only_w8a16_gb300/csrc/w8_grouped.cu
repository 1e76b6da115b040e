// w8_grouped.cu -- each group's rows times the group's plane:
//     y[i][n] = bf16( scale[n] sum_k W_g[n][k] x[i][k] ),  i in group g,
// or bf16(silu(gate) up) of a merged plane's row pairs.
//
// Pairs of CTAs (clusters of two SMs, one pair to every two SMs) walk over the
// items, static and in turn: an item is 256 rows of a group's plane by up to
// 256 of its positions, over all of k.  The product runs on tcgen05 over the
// pair (cta_group::2): each CTA widens its 128 rows of the weights into its
// tensor memory (operand A) and copies half of the positions' x (operand B),
// which the tensor cores of both read.  A CTA with 256 positions of its own
// would take 80 bytes a cycle from L2 at full rate, where an SM gets about 50;
// a pair's take 47 each.
//
// Twenty-four warps a CTA:
//   0-7   widen the weights: a stage is 128 or 256 columns of k; warps 0-3 take the
//         even stages, 4-7 the odd ones, each the 32 rows that it reaches in
//         tensor memory (two row tiles of the packed layout);
//   8-19  output: 32 rows by 16 positions at a time, from tensor memory;
//   20    copies the packed weights (boxes of a tensor map);
//   21    issues the steps (the pair's first CTA only);
//   22-23 copy the rows of x that the positions name into the K-major,
//         128-byte-swizzled layout.
// Tensor memory: the sums in two parts, of two items in turn or both of one, and
// the stages of A behind them.  The rings (weights; A and x) run on across items.
//
// Bound: few rows a group, the planes' bytes; many, the tensor cores' rate (or the
// power limit).  64 planes of 4096 x 6144 E4M3 (1.6 GB):
//   2 rows each, SiLU    255 us  6.3 TB/s of HBM (bf16 planes 7.2), tensor cores 16 %
//                                of the time
//   128 rows each, SiLU  365 us  1.13 PFLOP/s: a pair's 14 items of 48 stages, about
//                                1075 cycles a stage.  Its steps take 512 (8 of 256 x
//                                128 x 16 a pair), the widening alone 447 a CTA: what a
//                                stage waits for besides is not known
//   512 rows each        900 us  1.83 PFLOP/s, near the measured rate of the tensor cores
// and 64 of 6144 x 2048 with 256 rows each 296 us, 1.39 PFLOP/s: the tensor cores stand
// still while an item of more than 128 positions is stored, which has both parts of
// the sums.  Few planes (8 of 4096 x 6144 make 128 items, two rounds of the 76 pairs)
// are bound by what one pair takes in, a stage of 256 columns in 1240 cycles: 42 us
// where their bytes take 30.
//
// The tensor cores' fp32 sums cut off what does not fit instead of rounding it, as
// they do in a library's bf16 product: at 2048 columns 0.11 % of the outputs are the
// bf16 value next to the one that the exact sum rounds to, at 6144 0.34 %, as many as
// the library's (with every addition rounded to fp32: 0.03 and 0.05 %).
//
// Every wait is bounded; one that gave up sets the status word, and each copying
// warp waits for its own copies before the CTA leaves.
#include <stddef.h>

#include <type_traits>
#include <utility>

#include "w8_grouped_internal.h"
#include "w8_internal.h"
#include "w8_sum_parts.h"
#include "w8_tcgen.cuh"
#include "w8_turns.h"

namespace w8 {

__device__ int g_grouped_status;

namespace {

using namespace tcg;

constexpr int kConvWarps = 8, kOutWarps = 12;
constexpr int kXWarps = 2;
constexpr int kWarpWeights = kConvWarps + kOutWarps, kWarpIssue = kWarpWeights + 1, kWarpX = kWarpWeights + 2;
constexpr int kGpThreads = (kWarpX + kXWarps) * 32;
constexpr int kRings = 208 * 1024;        // weight and x stages
constexpr int kSmem = kRings + 1024;
constexpr int kTmem = 512;
constexpr int kMaxW = 7, kMaxX = 7, kMaxA = 7;
constexpr int kBox = 8 * 2048;            // bytes of a box of weights: 2 KB of each of 8 row tiles

constexpr int run_bytes(bool fp8) { return fp8 ? kRunFp8 : kRunBf16; }

// How many positions an item has at most, and the stages that leaves room for: of
// weights and x in shared memory, of A in tensor memory beside the sums.
struct Stages {
    int most;
    int blocks;  // K blocks (32 columns) of a stage
    int w, x, a; // stages of the rings
    int box;     // rows of a copy of x, where the positions are rows in turn
};
constexpr Stages kStagesOf[2][3] = {
    {{64, 4, 4, 7, 4, 16}, {128, 4, 3, 6, 3, 32}, {256, 4, 3, 3, 3, 32}}, // bf16
    {{64, 8, 5, 3, 3, 16}, {128, 4, 7, 6, 4, 32}, {256, 4, 5, 4, 4, 32}} // FP8
};
// The sums lie in two parts, one for each of two items in turn, so that one is
// read while the next item's are made; an item of more positions takes both.
constexpr int part_cols(const Stages &s) { return s.most < 128 ? s.most : 128; }
constexpr int stage_w(bool fp8, const Stages &s) { return 8 * s.blocks * run_bytes(fp8); }
constexpr int stage_x(const Stages &s) { return s.most / 2 * s.blocks * 64; }
constexpr bool fits(int fp8, int i)
{
    const Stages &s = kStagesOf[fp8][i];
    // (w and x >= a: see the widening warps)
    return s.w * stage_w(fp8, s) + s.x * stage_x(s) <= kRings && 2 * part_cols(s) + 16 * s.blocks * s.a <= kTmem && s.w >= s.a &&
           s.x >= s.a && s.w <= kMaxW && s.x <= kMaxX && s.a <= kMaxA && s.blocks % 4 == 0;
}
static_assert(fits(0, 0) && fits(0, 1) && fits(0, 2) && fits(1, 0) && fits(1, 1) && fits(1, 2), "stages");

struct Shared {
    uint64_t full_w[kMaxW], empty_w[kMaxW];
    uint64_t full_x[kMaxX], free_x[kMaxX];
    uint64_t ready[kMaxA], used[2 * kMaxA]; // A and x of a stage are in place (both CTAs'; in the first), A is used
    uint64_t sums[2], sums_read[2], end; // of the two parts
    int start[W8_MAX_GROUPS + 1];     // first position of each group
    int tiles[W8_MAX_GROUPS];         // position tiles up to and with each group
    int scan[kGpThreads / 32];
    uint32_t tmem;
};
static_assert(kSmem + sizeof(Shared) <= 227 * 1024, "shared memory");

// Waits for the last use of every slot, on `round` barriers (one a slot, if not said).
__device__ __forceinline__ bool wait_last(uint64_t *bars, int slots, int uses, int round = 0)
{
    bool ok = true;
    round = round ? round : slots;
    for (int i = max(uses - slots, 0); i < uses; ++i)
        ok = bar_wait(&bars[i % round], uint32_t(i / round) & 1u) && ok;
    return ok;
}

// ---- what passes between the two CTAs ------------------------------------------
__device__ __forceinline__ uint32_t in_first(const void *p)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
    return r;
}
// Arrive at a barrier of the first CTA.  What passes this way lies in tensor
// memory and in the async proxy's view of shared memory, completed before.
__device__ __forceinline__ void pair_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pair_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A rows 0 .. 127 in the first CTA's tensor memory, 128 .. 255 in the second's,
// each half of B in its CTA.
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

// Whether the phase of the given parity has ended, without waiting for it.
__device__ __forceinline__ bool bar_done(uint64_t *bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return done;
}

// A warp's wait.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, bar_wait(bar, parity));
}

// ---- copies ---------------------------------------------------------------------
// Arrive on the barrier once this thread's copies so far have landed.
__device__ __forceinline__ void copy16_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// 16 bytes global -> shared, `bytes` of them read and the others zero.
__device__ __forceinline__ void copy_part(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// ---- the widened A operand --------------------------------------------------------
// tcgen05.st 16x256b.x4: 16 lanes x 32 columns; registers 8j .. 8j+7 are block
// j's columns 2t, 2t+1 (of each step) of rows g and g+8.
__device__ __forceinline__ void store_a(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                 "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
// Units t and t+4 (four columns each) of rows g and g+8 of one packed run in
// shared memory, which lie in packed lanes 4g + t/2 and 4g + t/2 + 2.
template <bool kFp8> struct Units;
template <> struct Units<true> {
    uint32_t u0, u1, v0, v1;
    __device__ __forceinline__ void load(uint32_t run, int g, int t)
    {
        const uint32_t at = run + uint32_t((4 * g + (t >> 1)) * 16 + (t & 1) * 8);
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(u0), "=r"(u1) : "r"(at));
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v0), "=r"(v1) : "r"(at + 32));
    }
    __device__ __forceinline__ void widen(uint32_t *r) const
    {
        r[0] = widen_e4m3x2<kSelRowG>(u0);
        r[1] = widen_e4m3x2<kSelRowG>(u1);
        r[2] = widen_e4m3x2<kSelRowG8>(u0);
        r[3] = widen_e4m3x2<kSelRowG8>(u1);
        r[4] = widen_e4m3x2<kSelRowG>(v0);
        r[5] = widen_e4m3x2<kSelRowG>(v1);
        r[6] = widen_e4m3x2<kSelRowG8>(v0);
        r[7] = widen_e4m3x2<kSelRowG8>(v1);
    }
};
template <> struct Units<false> {
    uint4 u, v;
    __device__ __forceinline__ void load(uint32_t run, int g, int t)
    {
        const uint32_t at = run + uint32_t((t & 1) * 512 + (4 * g + (t >> 1)) * 16);
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at));
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at + 32));
    }
    __device__ __forceinline__ void widen(uint32_t *r) const
    {
        r[0] = u.x;
        r[1] = u.z;
        r[2] = u.y;
        r[3] = u.w;
        r[4] = v.x;
        r[5] = v.z;
        r[6] = v.y;
        r[7] = v.w;
    }
};

// ---- items ------------------------------------------------------------------------
struct Item {
    int group;      // -1: no such item
    int rows;       // first packed row of the pair
    int from, count; // positions
    int n;          // the step's N: count, rounded up to 32
    int tiles;      // position tiles of the group
};

__device__ __forceinline__ int cut(int v, int most) { return min(max(v, 0), most); }

// Item `id`: groups in turn, their row blocks in turn, position tiles innermost
// (the second tile's weights are then in L2).  A whole warp asks.
__device__ __forceinline__ Item find(const Shared &sh, int groups, int blocks, int id, int lane)
{
    Item it;
    it.group = -1;
    it.rows = it.from = it.count = it.n = it.tiles = 0;
    if (id >= sh.tiles[groups - 1] * blocks)
        return it;
    const int want = id / blocks;
    // the run of 32 groups that holds it, then the group
    const int run = __popc(__ballot_sync(0xffffffffu, 32 * lane + 31 < groups && sh.tiles[min(32 * lane + 31, groups - 1)] <= want));
    const int g = 32 * run + __popc(__ballot_sync(0xffffffffu, 32 * run + lane < groups && sh.tiles[min(32 * run + lane, groups - 1)] <= want));
    const int before = g ? sh.tiles[g - 1] : 0;
    const int tiles = sh.tiles[g] - before, rest = id - before * blocks;
    const int block = rest / tiles, tile = rest - block * tiles;
    const int all = sh.start[g + 1] - sh.start[g];
    const int per = ((all + tiles - 1) / tiles + 31) & ~31; // tiles of about one size
    it.group = g;
    it.rows = block * 256;
    it.from = sh.start[g] + tile * per;
    it.count = min(per, all - tile * per);
    it.n = (it.count + 31) & ~31;
    it.tiles = tiles;
    return it;
}

// g / (1 + e^-g) u.  With h = e^(-|g| / 2), 1 + e^-|g| = 1 + h h lies in 1 .. 2, and
// for g < 0 the fraction's e^g is split between both factors: nothing overflows, and
// a gate far below 0 leaves what the definition gives as long as bf16 holds it
// (silu(-100) u for a large u, too).  CUDA's expf is within 2 units (2^-22), counted
// twice in h h and in the factors, at most half as much in 1 + h h; the reciprocal is
// within one, the sum and the four products within half a unit each: in all
// (2 + 1 + 0.5 + 5 / 4) 2^-22 < 2^-19.7 of the value.
__device__ __forceinline__ float silu_mul(float g, float u)
{
    const float h = expf(-0.5f * fabsf(g)), f = g < 0.0f ? h : 1.0f;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(h, h, 1.0f)));
    return g * r * f * (u * f);
}

template <bool kFp8, bool kSilu, int kSize>
__global__ void __launch_bounds__(kGpThreads, 1)
    grouped_kernel(const __grid_constant__ GroupedArgs p, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x)
{
    constexpr Stages cfg = kStagesOf[kFp8][kSize];
    constexpr int kRun = run_bytes(kFp8), kStageW = stage_w(kFp8, cfg), kStageX = stage_x(cfg);
    constexpr int kChunks = cfg.blocks / 2, kChunkX = cfg.most / 2 * 128; // 64 columns of a CTA's positions
    constexpr int kPart = part_cols(cfg), kACol = 2 * kPart;
    constexpr int kUsed = used_bars(cfg.a);                              // barriers of A's uses
    constexpr bool kSlots = kUsed == cfg.a;                              // they are the slots' (no counts of their own)
    constexpr int kBoxBlocks = 2048 / kRun;                              // K blocks of a box of weights
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ __align__(16) Shared sh;
    const w8_grouped &a = p.a;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = int(blockIdx.x & 1); // the cluster is two CTAs along x
    uint8_t *const s_w = s_dyn + ((1024u - (smem_addr(s_dyn) & 1023u)) & 1023u);
    uint8_t *const s_x = s_w + cfg.w * kStageW;
    if (tid == 0) {
        for (int i = 0; i < kMaxW; ++i) {
            bar_init(&sh.full_w[i], 1);
            bar_init(&sh.empty_w[i], 4);
        }
        for (int i = 0; i < kMaxX; ++i) {
            bar_init(&sh.full_x[i], a.x_rows ? 32 * kXWarps : 2);
            bar_init(&sh.free_x[i], 1);
        }
        for (int i = 0; i < kMaxA; ++i) {
            bar_init(&sh.ready[i], 2 * 4);
            bar_init(&sh.used[2 * i], 1);
            bar_init(&sh.used[2 * i + 1], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.sums[i], 1);
            bar_init(&sh.sums_read[i], 2 * kOutWarps);
        }
        bar_init(&sh.end, 1);
        bar_init_fence();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_launch_dependents();
    pdl_wait();
    // ---- where each group begins, and its position tiles ---------------------------
    {
        constexpr int kPer = (W8_MAX_GROUPS + kGpThreads - 1) / kGpThreads;
        const int g0 = tid * kPer;
        // the largest offset so far: offsets that decrease name no position twice
        int top[kPer], inc = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int g = g0 + i;
            inc = max(inc, g <= a.n_groups ? cut(__ldg(a.offsets + g), a.n_rows) : 0);
            top[i] = inc;
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            inc = lane >= d ? max(inc, o) : inc;
        }
        if (lane == 31)
            sh.scan[warp] = inc;
        __syncthreads();
        int before = __shfl_up_sync(0xffffffffu, inc, 1);
        before = max(lane ? before : 0, int(__reduce_max_sync(0xffffffffu, lane < warp ? uint32_t(sh.scan[lane]) : 0u)));
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (g0 + i <= a.n_groups)
                sh.start[g0 + i] = max(top[i], before);
        __syncthreads();
        int sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int g = g0 + i;
            sum += g < a.n_groups ? (sh.start[g + 1] - sh.start[g] + cfg.most - 1) / cfg.most : 0;
            top[i] = sum;
        }
        inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            inc += lane >= d ? o : 0;
        }
        if (lane == 31)
            sh.scan[warp] = inc;
        __syncthreads();
        inc += int(__reduce_add_sync(0xffffffffu, lane < warp ? uint32_t(sh.scan[lane]) : 0u)) - sum;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (g0 + i < a.n_groups)
                sh.tiles[g0 + i] = inc + top[i];
    }
    fence_before();
    __syncthreads();
    pair_sync(); // both CTAs' barriers are ready, and both have their tensor memory
    fence_after();
    constexpr uint32_t tmem = 0; // all columns are this kernel's
    const int blocks = (p.rt + 15) / 16, pairs = int(gridDim.x >> 1);
    const int stages = (p.kb + cfg.blocks - 1) / cfg.blocks;
    bool ok = true;
    int id = int(blockIdx.x >> 1);
    auto item = [&] { return find(sh, a.n_groups, blocks, id, lane); };

    if (warp == kWarpWeights) {
        Turn to;
        const uint64_t first = policy_first(), normal = policy_normal();
        for (Item it = item(); it.group >= 0 && ok; id += pairs, it = item()) {
            const int tile0 = it.rows / kTileN + 8 * rank;
            const uint64_t policy = it.tiles > 1 ? normal : first; // read again by the group's other tiles, or not
            uint32_t who;
            if (elect_one(who)) {
                for (int st = 0; st < stages; ++st) {
                    if (to.n >= cfg.w)
                        ok = bar_wait(&sh.empty_w[to.k], to.parity ^ 1u);
                    if (!ok)
                        break;
                    const int boxes = (min(p.kb - st * cfg.blocks, cfg.blocks) + kBoxBlocks - 1) / kBoxBlocks;
                    bar_expect(&sh.full_w[to.k], uint32_t(boxes * kBox));
                    const uint32_t dst = smem_addr(s_w + to.k * kStageW);
                    for (int c = 0; c < boxes; ++c)
                        copy_box(dst + uint32_t(c * kBox), &map_w, (st * cfg.blocks / kBoxBlocks + c) * 256, tile0, it.group,
                                 &sh.full_w[to.k], policy);
                    to.step(cfg.w);
                }
            }
            __syncwarp();
            ok = __shfl_sync(0xffffffffu, ok, who);
            to.n = __shfl_sync(0xffffffffu, to.n, who);
            to.k = __shfl_sync(0xffffffffu, to.k, who);
            to.parity = __shfl_sync(0xffffffffu, to.parity, who);
        }
        ok = wait_last(sh.full_w, cfg.w, to.n) && ok;
    } else if (warp >= kWarpX) {
        // ---- x: rows that the positions name -> the K-major, 128-byte-swizzled layout ----
        const int h = warp - kWarpX;
        Turn to;
        const uint32_t x0 = smem_addr(s_x);
        for (Item it = item(); it.group >= 0 && ok; id += pairs, it = item()) {
            // this CTA's half of the positions; slots past them keep what they held: they
            // meet sums that nobody reads
            const int half = it.n / 2, mine = cut(it.count - rank * half, half), from = it.from + rank * half;
            if (!a.x_rows) {
                // rows in turn: boxes, each of two warps every second 64 of a stage's columns
                const int boxes = (mine + cfg.box - 1) / cfg.box;
                uint32_t who;
                if (h < 2 && elect_one(who)) {
                    for (int st = 0; st < stages; ++st) {
                        if (to.n >= cfg.x)
                            ok = bar_wait(&sh.free_x[to.k], to.parity ^ 1u);
                        if (!ok)
                            break;
                        const int chunks = (min(p.kb - st * cfg.blocks, cfg.blocks) + 1) / 2;
                        bar_expect(&sh.full_x[to.k], uint32_t((chunks - h + 1) / 2 * boxes * cfg.box * 128));
                        for (int c = h; c < chunks; c += 2)
                            for (int q = 0; q < boxes; ++q)
                                copy_box(x0 + uint32_t(to.k * kStageX + c * kChunkX + q * cfg.box * 128), &map_x,
                                         st * cfg.blocks * kTileK + 64 * c, from + q * cfg.box, &sh.full_x[to.k]);
                        to.step(cfg.x);
                    }
                }
                __syncwarp();
                if (h < 2) {
                    ok = __shfl_sync(0xffffffffu, ok, who);
                    to.n = __shfl_sync(0xffffffffu, to.n, who);
                    to.k = __shfl_sync(0xffffffffu, to.k, who);
                    to.parity = __shfl_sync(0xffffffffu, to.parity, who);
                }
                continue;
            }
            // Rows by number: 16 bytes a lane, eight lanes 64 columns of a row, a warp four
            // rows at a time, warp h rows 4 h + 8 i ..  (Gathering tensor-map copies, four
            // rows each, took 40 cycles a copy: 13 bytes a cycle, where 32 are needed.)
            constexpr int kRowsLane = cfg.most / 2 / (4 * kXWarps);
            const int r0 = 4 * h + (lane >> 3), c8 = lane & 7;
            const uint16_t *row[kRowsLane]; // zeros for a row outside: its sums are replaced
            uint32_t have = 0;
#pragma unroll
            for (int i = 0; i < kRowsLane; ++i) {
                row[i] = a.x + 8 * c8;
                if (r0 + 4 * kXWarps * i < mine) {
                    const int v = __ldg(a.x_rows + from + r0 + 4 * kXWarps * i);
                    have |= 1u << i;
                    if (v >= 0 && v < a.n_x)
                        row[i] += v * a.ldx;
                }
            }
            const uint32_t lane0 = x0 + uint32_t(r0 * 128 + ((c8 ^ (r0 & 7)) << 4));
            for (int st = 0; st < stages; ++st) {
                if (to.n >= cfg.x)
                    ok = warp_wait(&sh.free_x[to.k], to.parity ^ 1u);
                if (!ok)
                    break;
                const uint32_t dst = lane0 + uint32_t(to.k * kStageX);
                const int col = st * cfg.blocks * kTileK;
                if (col + cfg.blocks * kTileK <= p.k) {
#pragma unroll
                    for (int i = 0; i < kRowsLane; ++i)
                        if (have >> i & 1) {
#pragma unroll
                            for (int c = 0; c < kChunks; ++c)
                                copy16(dst + uint32_t(i * 512 * kXWarps + c * kChunkX), row[i] + col + 64 * c, true);
                        }
                } else { // the last columns: zeros past k
                    const int left = p.k - col - 8 * c8;
#pragma unroll
                    for (int i = 0; i < kRowsLane; ++i)
                        if (have >> i & 1) {
                            for (int c = 0; c < kChunks; ++c)
                                copy_part(dst + uint32_t(i * 512 * kXWarps + c * kChunkX), left > 64 * c ? row[i] + col + 64 * c : a.x,
                                          cut(2 * (left - 64 * c), 16));
                        }
                }
                copy16_arrive(&sh.full_x[to.k]);
                to.step(cfg.x);
            }
        }
        copy16_wait();
        const bool fine = ok;
        if (!a.x_rows && h < 2)
            ok = wait_last(sh.full_x, cfg.x, to.n) && ok;
        if (h == 0) {
            // The steps' last arrivals come to both CTAs, which may not leave before.
            if (fine)
                ok = wait_last(sh.free_x, cfg.x, to.n) && wait_last(sh.used, cfg.a, to.n, kUsed) && ok;
            ok = bar_wait(&sh.end, 0) && ok;
        }
    } else if (warp == kWarpIssue) {
        if (rank == 0) {
            const uint64_t b0 = desc128_k(smem_addr(s_x), 1024);
            Turn ta;              // of A
            int kx = 0, ku = 0;   // slot of x, barrier of A's use
            Parts parts;
            for (Item it = item(); it.group >= 0 && ok; id += pairs, it = item()) {
                parts.take(it.n, kPart);
                auto steps = [&](auto size) {
                    const uint32_t idesc = inst_desc(256, size, false, false);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (parts.frees(i))
                            ok = ok && bar_wait(&sh.sums_read[i], parts.free_parity(i));
                    const uint32_t sums = parts.first() * kPart;
                    bool there = false; // the stage was seen to be ready while the one before was issued
                    for (int st = 0; st < stages && ok; ++st) {
                        if (!there)
                            ok = bar_wait(&sh.ready[ta.k], ta.parity);
                        if (!ok)
                            break;
                        fence_after();
                        const uint64_t b = b0 + uint64_t((kx * kStageX) >> 4);
                        const uint32_t at = uint32_t(kACol + ta.k * 16 * cfg.blocks);
                        const int use = kSlots ? ta.k : ku, nb = p.kb - st * cfg.blocks;
                        ta.step(cfg.a);
                        there = bar_done(&sh.ready[ta.k], ta.parity);
                        for (int c = 0; c < kChunks; ++c) {
                            if (2 * c >= nb)
                                break;
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                if (q < 2 || 2 * c + 1 < nb)
                                    pair_mma_ts(sums, at + uint32_t(c * 32 + q * 8), b + uint64_t((c * kChunkX + q * 32) >> 4), idesc,
                                                uint32_t(st | c | q));
                        }
                        pair_commit(&sh.used[use]);
                        if constexpr (!kSlots)
                            ku = ku + 1 == kUsed ? 0 : ku + 1;
                        pair_commit(&sh.free_x[kx]);
                        kx = kx + 1 == cfg.x ? 0 : kx + 1;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (ok && parts.fills(i))
                            pair_commit(&sh.sums[i]);
                };
                uint32_t who;
                if (elect_one(who)) {
                    // For few positions a step takes less than its issue, which is
                    // shorter for an N that the compiler knows.
                    if (cfg.most > 64)
                        steps(it.n);
                    else if (it.n == 32)
                        steps(std::integral_constant<int, 32>{});
                    else
                        steps(std::integral_constant<int, 64>{});
                }
                __syncwarp();
                parts.done();
                ok = __shfl_sync(0xffffffffu, ok, who);
                kx = __shfl_sync(0xffffffffu, kx, who);
                if constexpr (!kSlots)
                    ku = __shfl_sync(0xffffffffu, ku, who);
                ta.k = __shfl_sync(0xffffffffu, ta.k, who);
                ta.parity = __shfl_sync(0xffffffffu, ta.parity, who);
            }
            // nothing is in the tensor cores when the CTAs free their memory
            if (elect_one())
                pair_commit(&sh.end);
            __syncwarp();
            ok = bar_wait(&sh.end, 0) && ok;
        }
    } else if (warp < kConvWarps) {
        // ---- weights: shared memory -> widened A --------------------------------------
        const int quarter = warp & 3, turn = warp >> 2;
        const int g = lane >> 2, t = lane & 3;
        const uint32_t at0 = tmem + (uint32_t(32 * quarter) << 16) + uint32_t(kACol);
        const uint32_t ready0 = in_first(&sh.ready[0]);
        // A barrier's phase may be waited for only once the one before has ended.  The
        // two turns run apart; that A's stage s - cfg.a is used (of whose barriers each
        // turn sees every phase: w8_turns.h) says that all its operands and those before
        // had come, so a turn waits for that first, and the rings of weights and x have at
        // least as many slots.
        Turn ta, tu, tw, tx; // tu: the use of the stage cfg.a before (unless kSlots)
        for (Item it = item(); it.group >= 0 && ok; id += pairs, it = item()) {
            for (int st = 0; st < stages; ++st) {
                if ((ta.n & 1) == turn) {
                    auto wait = [&](uint64_t *bar, uint32_t parity) { return warp_wait(bar, parity); };
                    if (ta.n >= cfg.a)
                        ok = kSlots ? wait(&sh.used[ta.k], ta.parity ^ 1u) : wait(&sh.used[tu.k], tu.parity);
                    ok = ok && wait(&sh.full_w[tw.k], tw.parity);
                    if (!ok)
                        break;
                    // Two blocks of a row tile at a time, in a loop of two: longer code
                    // does not stay in the instruction cache beside the other roles'.
                    const uint32_t w0 = smem_addr(s_w + tw.k * kStageW + 2 * quarter * 2048);
                    auto pair_at = [](int i) { // tile i % 2, blocks 2 (i / 2), + 1
                        constexpr int kPairs = kBoxBlocks / 2;
                        return uint32_t((i & 1) * 2048 + (i >> 1) / kPairs * kBox + (i >> 1) % kPairs * 2 * kRun);
                    };
                    Units<kFp8> w[2];
                    w[0].load(w0, g, t);
                    w[1].load(w0 + kRun, g, t);
                    fence_after();
                    const int todo = (min(p.kb - st * cfg.blocks, cfg.blocks) + 1) & ~1;
#pragma unroll 2
                    for (int i = 0; i < todo; ++i) {
                        uint32_t r[16];
                        w[0].widen(r);
                        w[1].widen(r + 8);
                        if (i + 1 < todo) {
                            const uint32_t from = w0 + pair_at(i + 1);
                            w[0].load(from, g, t);
                            w[1].load(from + kRun, g, t);
                        }
                        store_a(at0 + (uint32_t((i & 1) * 16) << 16) + uint32_t(ta.k * 16 * cfg.blocks + (i >> 1) * 32), r);
                    }
                    // (only now: the stores have taken the loads' results, and an arrival
                    // right behind the loads let copies overwrite what they were to read)
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(&sh.empty_w[tw.k]);
                    wait_st();
                    fence_before();
                    // x of the stage has landed here, too: one arrival says both
                    ok = wait(&sh.full_x[tx.k], tx.parity);
                    if (!ok)
                        break;
                    fence_async_shared(); // (x that threads have copied, for the tensor cores)
                    __syncwarp();
                    if (lane == 0)
                        pair_arrive(ready0 + uint32_t(8 * ta.k));
                }
                if constexpr (!kSlots)
                    if (ta.n >= cfg.a)
                        tu.step(kUsed);
                ta.step(cfg.a);
                tw.step(cfg.w);
                tx.step(cfg.x);
            }
        }
    } else {
        // ---- output: 32 rows, 16 positions at a time, every third such run -----------------
        constexpr int kTeams = kOutWarps / 4;
        const int quarter = warp & 3, team = (warp - kConvWarps) >> 2;
        const uint32_t read_bar = in_first(&sh.sums_read[0]);
        const bool odd = lane & 1, up = lane & 8;
        Parts parts;
        for (Item it = item(); it.group >= 0 && ok; id += pairs, it = item()) {
            parts.take(it.n, kPart);
            const int row = it.rows + 128 * rank + 32 * quarter + lane;
            const float scale = kFp8 && row < p.n ? __ldg(p.scale + it.group * p.scale_step + row) : 1.0f;
            // where 16 of the positions go, a lane each, and whether their row of x is outside
            auto target = [&](int c, bool &zero) {
                const int i = 16 * c + (lane & 15);
                zero = false;
                if (i >= it.count)
                    return -1;
                const int at = it.from + i;
                const int r = a.y_rows ? __ldg(a.y_rows + at) : at, x = a.x_rows ? __ldg(a.x_rows + at) : at;
                zero = x < 0 || x >= a.n_x;
                return r >= 0 && r < a.n_y ? r : -1;
            };
            bool zero;
            int to = target(team, zero);
            // A lane stores two neighbouring columns of a position: its own and lane ^ 1's.
            // With SiLU the lanes of gate rows (up rows are 8 lanes on) store those of one
            // position, the lanes of up rows the same columns of the next.
            const int first = (row & ~1) - (kSilu && up ? 8 : 0);
            uint16_t *const y = a.y + (kSilu ? out_col(first, true, p.half) : out_col(first, p.act != kActPlain, p.half));
            const bool held = first < p.n, both = first + 1 < p.n;
            auto store = [&](int r, uint32_t v) {
                if (held && r >= 0) {
                    uint16_t *const at = y + r * a.ldy;
                    if (both && p.wide_y) {
                        *reinterpret_cast<uint32_t *>(at) = v;
                    } else {
                        at[0] = uint16_t(v);
                        if (both)
                            at[1] = uint16_t(v >> 16);
                    }
                }
            };
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (parts.fills(i))
                    ok = ok && warp_wait(&sh.sums[i], parts.fill_parity(i));
            if (!ok)
                break;
            fence_after();
            const uint32_t d0 = tmem + (uint32_t(32 * quarter) << 16) + parts.first() * kPart;
            // In a loop that is not unrolled: eight times its code, run through once an
            // item, took the other roles' out of the instruction cache (3 to 5 us an item).
#pragma unroll 1
            for (int c = team; 16 * c < it.count || c == team; c += kTeams) {
                const bool last = 16 * (c + kTeams) >= it.count, some = 16 * c < it.count;
                float d[16];
                if (some)
                    ld32x16(d, d0 + uint32_t(16 * c));
                const uint32_t zeros = __ballot_sync(0xffffffffu, zero);
                const int now = to;
                to = target(c + kTeams, zero);
                wait_ld();
                if (last) { // another item's steps may begin here
                    fence_before();
                    __syncwarp();
                    if (lane == 0)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (parts.fills(i))
                                pair_arrive(read_bar + uint32_t(8 * i));
                }
                if (!some)
                    break;
                if (zeros) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        d[e] = zeros >> e & 1 ? 0.0f : d[e];
                }
                if constexpr (kFp8) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        d[e] *= scale;
                }
                if constexpr (kSilu) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        // of two positions the gate's lane takes the first, the up's the second
                        float h[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float mine = up ? d[e + 2 * k + 1] : d[e + 2 * k];
                            const float other = __shfl_xor_sync(0xffffffffu, up ? d[e + 2 * k] : d[e + 2 * k + 1], 8);
                            h[k] = silu_mul(up ? other : mine, up ? mine : other);
                        }
                        const float beside = __shfl_xor_sync(0xffffffffu, odd ? h[0] : h[1], 1);
                        const int r = __shfl_sync(0xffffffffu, now, e + (odd ? 2 : 0) + (up ? 1 : 0));
                        store(r, pack_bf16(odd ? beside : h[0], odd ? h[1] : beside));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float beside = __shfl_xor_sync(0xffffffffu, odd ? d[e] : d[e + 1], 1);
                        const int r = __shfl_sync(0xffffffffu, now, e + (odd ? 1 : 0));
                        store(r, pack_bf16(odd ? beside : d[e], odd ? d[e + 1] : beside));
                    }
                }
            }
            parts.done();
        }
    }
    if (!ok)
        atomicOr(&g_grouped_status, 1);
    fence_before();
    __syncthreads();
    pair_sync(); // neither CTA leaves while the other's steps or arrivals may reach it
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(kTmem) : "memory");
    }
}

// The groups' packed planes as [group][row tile][8 bytes], in boxes of 256 x 8 x 1.
bool encode_weight_map(CUtensorMap *map, const GroupedArgs &a, int run)
{
    const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
    if (!enc)
        return false;
    const cuuint64_t tile = cuuint64_t(a.kb) * cuuint64_t(run);
    const cuuint64_t dims[3] = {tile / 8, cuuint64_t(a.rt), cuuint64_t(a.a.n_groups)};
    const cuuint64_t strides[2] = {tile, a.a.n_groups > 1 ? cuuint64_t(a.wp_step) : tile * cuuint64_t(a.rt)};
    const cuuint32_t box[3] = {256, 8, 1}, one[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, 3, const_cast<uint8_t *>(a.wp), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kFp8, bool kSilu, int kSize>
cudaError_t launch(const GroupedArgs &a, int sms, cudaStream_t s)
{
    auto *fn = &grouped_kernel<kFp8, kSilu, kSize>;
    constexpr Stages cfg = kStagesOf[kFp8][kSize];
    CUtensorMap map, map_w;
    if (!encode_weight_map(&map_w, a, run_bytes(kFp8)))
        return cudaErrorInvalidValue;
    const uint64_t sizes[2] = {uint64_t(a.k), uint64_t(a.a.n_x)}, strides[1] = {uint64_t(a.a.ldx) * 2};
    const uint32_t box[2] = {64, uint32_t(cfg.box)}; // (unused where rows go by number)
    if (!encode_bf16_map(&map, a.a.x, 2, sizes, strides, box))
        return cudaErrorInvalidValue;
    // every group may end in a part of a tile
    const int64_t tiles = a.a.n_rows / cfg.most + (a.a.n_groups < a.a.n_rows ? a.a.n_groups : a.a.n_rows);
    const int64_t items = tiles * ((a.rt + 15) / 16);
    if (items > INT32_MAX)
        return cudaErrorInvalidValue;
    const int pairs = items < sms / 2 ? int(items) : sms / 2;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(unsigned(2 * pairs));
    lc.blockDim = dim3(kGpThreads);
    lc.dynamicSmemBytes = kSmem;
    lc.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 2;
    return cudaLaunchKernelEx(&lc, fn, a, map_w, map);
}

template <bool kFp8, bool kSilu>
cudaError_t launch_sized(const GroupedArgs &a, int sms, cudaStream_t s)
{
    // Positions of an item: more take the weights fewer times, fewer leave room for
    // more and longer stages.  The host knows a mean only, and groups are uneven as a
    // rule; rows of no group count in it, and groups without rows do, so that where
    // most rows lie elsewhere items are too large for what is here (at 32 rows 314 us
    // for 258), and where few of the groups are hit too small (128 rows, 491 for 364).
    // Items of up to 64 / 128 / 256, 64 planes of 4096 x 6144 E4M3, SiLU, us:
    //   rows a group      all alike          uneven (a twelfth to twice the mean)
    //   32             258 / 297 / 314             292 / 300 / 320
    //   48             267 / 301 / 322             345 / 303 / 324
    //   64             281 / 305 / 329             395 / 346 / 330
    //   96             488 / 316 / 346             504 / 396 / 355
    //   128            491 / 341 / 364             627 / 444 / 381
    // and of 6144 x 2048, uneven: 48 rows 204 / 183 / 186, 100 rows 312 / 254 / 211
    // (bf16 270 / 256 / 256 and 370 / 320 / 279).
    const int64_t groups = a.a.n_groups < a.a.n_rows ? a.a.n_groups : a.a.n_rows;
    return a.a.n_rows <= 40 * groups  ? launch<kFp8, kSilu, 0>(a, sms, s)
           : a.a.n_rows <= 60 * groups ? launch<kFp8, kSilu, 1>(a, sms, s)
                                      : launch<kFp8, kSilu, 2>(a, sms, s);
}

// Every kernel's limit, at the first call on a device.
template <int... kI> cudaError_t raise_all(std::integer_sequence<int, kI...>)
{
    static std::atomic<uint64_t> raised{0};
    return raise_smem(raised, {{reinterpret_cast<const void *>(&grouped_kernel<kI / 6 != 0, kI / 3 % 2 != 0, kI % 3>), kSmem}...});
}

} // namespace

cudaError_t launch_grouped(const GroupedArgs &a, bool fp8, int sms, cudaStream_t s)
{
    const cudaError_t e = raise_all(std::make_integer_sequence<int, 12>{});
    if (e != cudaSuccess)
        return e;
    if (a.act == kActSiluMul)
        return fp8 ? launch_sized<true, true>(a, sms, s) : launch_sized<false, true>(a, sms, s);
    return fp8 ? launch_sized<true, false>(a, sms, s) : launch_sized<false, false>(a, sms, s);
}

cudaError_t grouped_status(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_grouped_status, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_grouped_status, &zero, sizeof(int));
    }
    return e;
}

} // namespace w8
