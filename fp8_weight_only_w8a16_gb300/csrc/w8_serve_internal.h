// w8_serve_internal.h -- what the C-ABI layer of the serving operators
// (w8_serve_api.cu) hands to their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <initializer_list>

#include "w8_serve.h"

namespace w8 {

struct TableArgs {
    const int32_t *ctx, *fresh, *free_pages, *free_head;
    int32_t *table, *seq_lens, *cu, *positions, *head_out, *status;
    int64_t *slots;
    int64_t ld_table;
    int n_req, page, n_free, max_pages, max_tok;
};
cudaError_t launch_block_tables(const TableArgs &a, int sms, cudaStream_t s);

struct CacheWriteArgs {
    const uint16_t *latent, *rope;
    int64_t ld_latent, ld_rope;
    const int64_t *slots;
    uint16_t *cache;
    int64_t ld_page, ld_tok, n_slots;
    int page, n_tok;
};
cudaError_t launch_cache_write(const CacheWriteArgs &a, cudaStream_t s);

cudaError_t launch_latent_paged(const w8_latent_paged &a, void *ws, int sms, cudaStream_t s);
size_t latent_paged_ws_bytes(int n_tok, int n_heads, int n_req, int sms);

cudaError_t launch_latent_expanded(const w8_latent_expanded &a, int sms, cudaStream_t s);
cudaError_t launch_expanded_pairs(const w8_latent_expanded &a, cudaStream_t s); // its kernel for pairs of CTAs

// Logits of one row go to `splits` CTAs; their partial results meet in the
// workspace: a head of kLogprobsCounters arrival counters, one a row, always
// at the same place, then one LogprobsPart a (row, split).
constexpr int kLogprobsCounters = 8192;
struct LogprobsPart {
    float m, z, w;      // running maximum, sum, sum of p ln p (relative to m)
    uint32_t pad;
    uint64_t key[W8_MAX_TOP];
};
struct LogprobsArgs {
    const void *x;
    int64_t ld;
    int rows, vocab, top, splits;
    const int32_t *tokens;
    float *logprob, *entropy, *top_logprobs;
    int32_t *top_ids;
    int *counters;
    LogprobsPart *parts;
};
int logprobs_splits(int rows, int vocab, int sms);
cudaError_t launch_logprobs(const LogprobsArgs &a, bool bf16, cudaStream_t s);

// The attention kernels' status words (w8_serve_device_status): not 0 once a
// wait gave up.
cudaError_t paged_status(int *out, bool reset);
cudaError_t expanded_status(int *out, bool reset);
cudaError_t pairs_status(int *out, bool reset);

// Raise a kernel's dynamic shared-memory limit, once a device (`done`: a bit a
// device; devices past 63 raise it every time).
inline cudaError_t raise_smem(std::atomic<uint64_t> &done, const void *fn, int bytes)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)))
        return e;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64)
        done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    return e;
}

// ... of all kernels of an operator, whichever of them the call goes to: a capture
// that comes after one call of the operator sets no attribute.
struct SmemLimit {
    const void *fn;
    int bytes;
};
inline cudaError_t raise_smem(std::atomic<uint64_t> &done, std::initializer_list<SmemLimit> kernels)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)))
        return e;
    for (const SmemLimit &k : kernels) {
        e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.bytes);
        if (e != cudaSuccess)
            return e;
    }
    if (dev < 64)
        done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    return cudaSuccess;
}

// Launch with the programmatic-dependency attribute (the kernel waits for the
// stream's previous kernel itself, before its first global access).
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*fn)(P...), dim3 grid, int block, size_t smem, cudaStream_t s,
                                    const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, P(args)...);
}

} // namespace w8
