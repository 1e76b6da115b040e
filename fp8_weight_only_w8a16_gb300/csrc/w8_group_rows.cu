// w8_group_rows.cu -- rows by their groups: a stable counting sort of up to
// 1024 groups.
//
// A CTA ranks one chunk of the items.  Its warps hold consecutive segments of
// the chunk; each counts its segment's groups in a histogram of its own (32
// items at a time, the lanes of one group found by match: no atomics, so the
// order is always the same).  The histograms are then summed down the warps
// and over the groups, which gives each warp the place of its first item of
// each group, and a second walk through the segment writes the items there.
// Several chunks: a first launch writes each chunk's counts, the second adds
// those of the chunks before.
//
// Bound: latency, the chains of loads and matches (12 to 16 bytes an item are
// nothing: 0.2 us for 98304 items).  512 items of 256 groups 7 us; 98304 of 128
// groups in 96 chunks 6 us to count and 14 to place, launches apart.
#include <atomic>

#include "w8_device.cuh"
#include "w8_grouped_internal.h"

namespace w8 {
namespace {

constexpr int kGrThreads = 1024;
constexpr int kGrWarps = kGrThreads / 32;

struct Segment {
    int from, to;
};
__device__ __forceinline__ Segment segment(const GroupArgs &a, int warp)
{
    const int c0 = min(int64_t(blockIdx.x) * a.chunk, int64_t(a.n)), c1 = min(int64_t(c0) + a.chunk, int64_t(a.n));
    const int per = ((c1 - c0 + kGrWarps - 1) / kGrWarps + 31) & ~31;
    const int from = min(int64_t(c0) + int64_t(warp) * per, int64_t(c1));
    return {from, int(min(int64_t(from) + per, int64_t(c1)))};
}

// A lane's item: its group (-1: of none) and the lanes with items of that group.
struct Found {
    int g;
    uint32_t same;
};
__device__ __forceinline__ Found find(const GroupArgs &a, Segment s, int it)
{
    int g = it < s.to ? __ldg(a.ids + it) : -1;
    if (g < 0 || g >= a.groups)
        g = -1;
    return {g, __match_any_sync(0xffffffffu, g)};
}

// Calls f(item, group, lanes of that group) for the segment's items in turn,
// by whole warps; `first` is what was found of the first 32.
template <typename F>
__device__ __forceinline__ void walk(const GroupArgs &a, Segment s, int lane, Found first, F f)
{
    for (int i = s.from; i < s.to; i += 32) {
        const Found v = i == s.from ? first : find(a, s, i + lane);
        f(i + lane, v.g, v.same);
        __syncwarp();
    }
}

// Histograms of the chunk's warps, [warp][groups]; on return row w holds the
// counts of warps before w, and total[] the chunk's.
__device__ __forceinline__ void chunk_counts(const GroupArgs &a, Segment s, Found first, int *hist, int *total, int warp, int lane)
{
    for (int i = threadIdx.x; i < kGrWarps * a.groups; i += kGrThreads)
        hist[i] = 0;
    __syncthreads();
    int *mine = hist + warp * a.groups;
    walk(a, s, lane, first, [&](int, int g, uint32_t same) {
        if (g >= 0 && lane == __ffs(int(same)) - 1)
            mine[g] += __popc(same);
    });
    __syncthreads();
    for (int g = threadIdx.x; g < a.groups; g += kGrThreads) {
        int c[kGrWarps], sum = 0; // (all read before the first is written)
#pragma unroll
        for (int w = 0; w < kGrWarps; ++w)
            c[w] = hist[w * a.groups + g];
#pragma unroll
        for (int w = 0; w < kGrWarps; ++w) {
            hist[w * a.groups + g] = sum;
            sum += c[w];
        }
        total[g] = sum;
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kGrThreads) count_kernel(const GroupArgs a)
{
    extern __shared__ int s_hist[];
    __shared__ int total[W8_MAX_GROUPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const Segment s = segment(a, warp);
    chunk_counts(a, s, find(a, s, s.from + lane), s_hist, total, warp, lane);
    for (int g = threadIdx.x; g < a.groups; g += kGrThreads)
        a.counts[int64_t(blockIdx.x) * a.groups + g] = total[g];
}

__global__ void __launch_bounds__(kGrThreads) place_kernel(const GroupArgs a)
{
    extern __shared__ int s_hist[];
    __shared__ int base[W8_MAX_GROUPS];
    __shared__ int s_sum[kGrWarps];
    __shared__ int2 s_part[kGrThreads];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    static_assert(W8_MAX_GROUPS <= kGrThreads, "a thread a group");
    pdl_launch_dependents();
    pdl_wait();
    const Segment s = segment(a, warp);
    const Found first = find(a, s, s.from + lane);
    chunk_counts(a, s, first, s_hist, base, warp, lane);
    // group tid: items of it in all, and in the chunks before
    int all = 0, before = 0;
    if (a.chunks == 1) {
        if (tid < a.groups)
            all = base[tid];
    } else {
        // several threads a group, each every so many chunks
        const int stripes = min(kGrThreads / a.groups, 32), mine = tid / a.groups, g = tid - mine * a.groups;
        if (mine < stripes) {
#pragma unroll 16
            for (int c = mine; c < a.chunks; c += stripes) {
                const int v = __ldcg(a.counts + int64_t(c) * a.groups + g);
                before += c < int(blockIdx.x) ? v : 0;
                all += v;
            }
            s_part[tid] = make_int2(all, before);
        }
        __syncthreads();
        all = before = 0;
        if (tid < a.groups)
            for (int i = 0; i < stripes; ++i) {
                const int2 v = s_part[i * a.groups + tid];
                all += v.x;
                before += v.y;
            }
    }
    int inc = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        inc += lane >= d ? o : 0;
    }
    if (lane == 31)
        s_sum[warp] = inc;
    __syncthreads(); // (and every thread has read its base)
    int held = 0;
#pragma unroll
    for (int w = 0; w < kGrWarps; ++w) {
        const int v = s_sum[w];
        inc += w < warp ? v : 0;
        held += v;
    }
    if (tid < a.groups) {
        base[tid] = inc - all + before;
        if (blockIdx.x == 0)
            a.offsets[tid + 1] = inc;
    }
    if (blockIdx.x == 0 && tid == 0)
        a.offsets[0] = 0;
    __syncthreads();
    int *mine = s_hist + warp * a.groups;
    walk(a, s, lane, first, [&](int it, int g, uint32_t same) {
        const int at = g >= 0 ? base[g] + mine[g] + __popc(same & ((1u << lane) - 1)) : 0;
        __syncwarp();
        if (g >= 0 && lane == __ffs(int(same)) - 1)
            mine[g] += __popc(same);
        if (g >= 0) {
            a.order[at] = it;
            if (a.rows)
                a.rows[at] = it / a.per;
        }
    });
    // behind the last group's items
    for (int64_t j = int64_t(held) + int64_t(blockIdx.x) * kGrThreads + tid; j < a.n; j += int64_t(gridDim.x) * kGrThreads) {
        a.order[j] = -1;
        if (a.rows)
            a.rows[j] = -1;
    }
}

} // namespace

cudaError_t launch_group_rows(const GroupArgs &a, cudaStream_t s)
{
    static std::atomic<uint64_t> raised{0};
    const size_t smem = size_t(kGrWarps) * size_t(a.groups) * sizeof(int);
    constexpr int most = kGrWarps * W8_MAX_GROUPS * int(sizeof(int));
    cudaError_t e = raise_smem(raised, {{reinterpret_cast<const void *>(&place_kernel), most},
                                        {reinterpret_cast<const void *>(&count_kernel), most}});
    if (e != cudaSuccess)
        return e;
    if (a.chunks > 1) {
        e = launch_dependent(count_kernel, dim3(unsigned(a.chunks)), kGrThreads, smem, s, a);
        if (e != cudaSuccess)
            return e;
    }
    return launch_dependent(place_kernel, dim3(unsigned(a.chunks)), kGrThreads, smem, s, a);
}

} // namespace w8
