// w8_paging.cu -- the paged bookkeeping of a serving step (block tables, slot
// map) and the latent-cache write.
#include <cuda_runtime.h>
#include <stdint.h>

#include "w8_device.cuh"
#include "w8_serve_internal.h"

namespace w8 {

namespace {

constexpr int kTableThreads = 1024;

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d)
            v += o;
    }
    return v;
}

// Block tables and slot map (definition in w8_serve.h).  The work is two
// prefix sums over the requests, then one independent answer a page and a
// token.  Every CTA makes the prefix sums of all requests for itself, into
// shared memory: at most 16384 requests are 128 KB of lengths from L2, and
// the CTAs then need no word from one another -- one launch, no grid-wide
// wait.  A fresh page's number comes straight from the free list for the
// table entry and for its tokens alike, so no token waits for a table entry
// that another CTA writes.  Bound by latency: a launch, two dependent loads
// (lengths, free list) and the scan.  64 requests of one token 3.9 us, 1021 with
// 130,000 tokens 5.3 us (replayed).
__global__ void __launch_bounds__(kTableThreads) block_tables_kernel(const TableArgs a)
{
    extern __shared__ int32_t s_tab[]; // cu [n_req + 1], page base [n_req], context [n_req]
    __shared__ int64_t s_tok[32], s_page[32];
    __shared__ int s_bad;
    int32_t *const s_cu = s_tab, *const s_base = s_tab + a.n_req + 1, *const s_ctx = s_base + a.n_req;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int threads = blockDim.x, warps = threads >> 5;
    if (tid == 0)
        s_bad = 0;
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();

    // each thread's run of requests, its token and page sums
    const int per = (a.n_req + threads - 1) / threads;
    const int r0 = tid * per, r1 = r0 + per < a.n_req ? r0 + per : a.n_req;
    const int head = max(__ldg(a.free_head), 0);
    int64_t toks = 0, pages = 0;
    int bad = 0;
    for (int r = r0; r < r1; ++r) {
        int64_t ctx = __ldg(a.ctx + r), fresh = __ldg(a.fresh + r);
        if (ctx < 0 || fresh < 0 || ctx + fresh > INT32_MAX)
            bad |= 4;
        ctx = ctx < 0 ? 0 : ctx;
        fresh = fresh < 0 ? 0 : fresh;
        if (ctx + fresh > INT32_MAX)
            fresh = INT32_MAX - ctx;
        const int64_t have = (ctx + a.page - 1) / a.page, want = (ctx + fresh + a.page - 1) / a.page;
        if (want > a.max_pages)
            bad |= 2;
        s_ctx[r] = int32_t(ctx);
        s_cu[r] = int32_t(fresh); // the length, until the sums are known
        s_base[r] = int32_t(min(want, int64_t(a.max_pages)) - min(have, int64_t(a.max_pages)));
        toks += fresh;
        pages += s_base[r];
    }
    const int64_t itoks = warp_scan(toks, lane), ipages = warp_scan(pages, lane);
    if (lane == 31) {
        s_tok[warp] = itoks;
        s_page[warp] = ipages;
    }
    if (bad)
        atomicOr(&s_bad, bad);
    __syncthreads();
    if (warp == 0) {
        const int64_t t = lane < warps ? s_tok[lane] : 0, p = lane < warps ? s_page[lane] : 0;
        const int64_t it = warp_scan(t, lane), ip = warp_scan(p, lane);
        s_tok[lane] = it;
        s_page[lane] = ip;
    }
    __syncthreads();
    const int64_t all_toks = s_tok[31], all_pages = s_page[31];
    int64_t tbase = itoks - toks + (warp ? s_tok[warp - 1] : 0);
    int64_t pbase = ipages - pages + (warp ? s_page[warp - 1] : 0) + head;
    for (int r = r0; r < r1; ++r) {
        const int32_t fresh = s_cu[r], need = s_base[r];
        const int32_t cut = int32_t(min(tbase, int64_t(INT32_MAX)));
        s_cu[r] = cut;
        s_base[r] = int32_t(min(pbase, int64_t(INT32_MAX)));
        if (blockIdx.x == 0) {
            a.seq_lens[r] = s_ctx[r] + fresh;
            a.cu[r] = cut;
        }
        tbase += fresh;
        pbase += need;
    }
    if (tid == 0) {
        const int32_t all = int32_t(min(all_toks, int64_t(INT32_MAX)));
        s_cu[a.n_req] = all;
        if (blockIdx.x == 0) {
            a.cu[a.n_req] = all;
            *a.head_out = int32_t(min(head + all_pages, int64_t(max(a.n_free, 0))));
            *a.status = s_bad | (head + all_pages > a.n_free ? 1 : 0) | (all_toks > a.max_tok ? 4 : 0);
        }
    }
    __syncthreads();

    // fresh table entries: a warp a request, the requests dealt over all CTAs
    for (int r = blockIdx.x * warps + warp; r < a.n_req; r += gridDim.x * warps) {
        const int32_t ctx = s_ctx[r], base = s_base[r];
        // (not from the offsets: they are cut at the end of the number range)
        const int64_t fresh = min(max(__ldg(a.fresh + r), 0), INT32_MAX - ctx);
        const int have = int((int64_t(ctx) + a.page - 1) / a.page);
        const int want = int(min((ctx + fresh + a.page - 1) / a.page, int64_t(a.max_pages)));
        for (int p = have + lane; p < want; p += 32) {
            const int64_t f = int64_t(base) + p - have;
            a.table[r * a.ld_table + p] = f < a.n_free ? __ldg(a.free_pages + f) : -1;
        }
    }
    // tokens: the request by bisection of cu, then its page
    for (int64_t t = int64_t(blockIdx.x) * threads + tid; t < a.max_tok; t += int64_t(gridDim.x) * threads) {
        int64_t slot = -1;
        int32_t pos = -1;
        if (t < s_cu[a.n_req]) {
            int lo = 0, hi = a.n_req; // cu[lo] <= t < cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_cu[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            pos = s_ctx[lo] + int32_t(t - s_cu[lo]);
            const int p = pos / a.page, have = int((int64_t(s_ctx[lo]) + a.page - 1) / a.page);
            int32_t entry = -1;
            if (p < a.max_pages) {
                const int64_t f = int64_t(s_base[lo]) + p - have;
                if (p < have)
                    entry = a.table[lo * a.ld_table + p];
                else if (f < a.n_free)
                    entry = __ldg(a.free_pages + f);
            }
            if (entry >= 0)
                slot = int64_t(entry) * a.page + pos % a.page;
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
}

// Latent-cache write: 72 vectors of 16 bytes a token (64 of the latent, 8 of
// the rope key), a thread four of them a block's width apart, all loads
// before the first store.  Nothing but the copy: bound by HBM when there are
// many tokens (16391: 6.3 us, 6.0 TB/s), by the launch when there are few (8:
// 1.9 us).
constexpr int kWriteThreads = 256, kWriteVecs = 4, kRowVecs = W8_LATENT_ROW / 8;

__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const CacheWriteArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t items = int64_t(a.n_tok) * kRowVecs;
    const int64_t i0 = int64_t(blockIdx.x) * (kWriteThreads * kWriteVecs) + threadIdx.x;
    uint4 v[kWriteVecs];
    uint16_t *dst[kWriteVecs];
#pragma unroll
    for (int k = 0; k < kWriteVecs; ++k) {
        const int64_t i = i0 + k * kWriteThreads;
        dst[k] = nullptr;
        if (i < items) {
            const int64_t t = i / kRowVecs;
            const int c = int(i - t * kRowVecs);
            const int64_t slot = __ldg(a.slots + t);
            if (slot >= 0 && slot < a.n_slots) {
                const int64_t page = slot / a.page;
                dst[k] = a.cache + page * a.ld_page + (slot - page * a.page) * a.ld_tok + 8 * c;
            }
            const uint16_t *src = c < W8_LATENT_DIM / 8 ? a.latent + t * a.ld_latent + 8 * c
                                                        : a.rope + t * a.ld_rope + 8 * (c - W8_LATENT_DIM / 8);
            v[k] = __ldg(reinterpret_cast<const uint4 *>(src));
        }
    }
#pragma unroll
    for (int k = 0; k < kWriteVecs; ++k)
        if (dst[k])
            *reinterpret_cast<uint4 *>(dst[k]) = v[k];
}

} // namespace

cudaError_t launch_block_tables(const TableArgs &a, int sms, cudaStream_t s)
{
    const size_t smem = (3 * size_t(a.n_req) + 1) * sizeof(int32_t);
    if (smem > 48 * 1024) {
        static std::atomic<uint64_t> raised{0};
        const cudaError_t e = raise_smem(raised, reinterpret_cast<const void *>(&block_tables_kernel),
                                         (3 * W8_MAX_REQUESTS + 1) * int(sizeof(int32_t)));
        if (e != cudaSuccess)
            return e;
    }
    // one CTA a 1024 tokens or requests' warps, one a SM at most
    const int64_t most = max(int64_t(a.max_tok), int64_t(a.n_req));
    const int64_t want = (most + kTableThreads - 1) / kTableThreads;
    const int grid = int(want < 1 ? 1 : want > sms ? sms : want);
    return launch_dependent(&block_tables_kernel, dim3(unsigned(grid)), kTableThreads, smem, s, a);
}

cudaError_t launch_cache_write(const CacheWriteArgs &a, cudaStream_t s)
{
    const int64_t per = kWriteThreads * kWriteVecs;
    const int64_t grid = (int64_t(a.n_tok) * kRowVecs + per - 1) / per;
    return launch_dependent(&cache_write_kernel, dim3(unsigned(grid)), kWriteThreads, 0, s, a);
}

} // namespace w8
