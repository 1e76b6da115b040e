// w8_grouped_internal.h -- what the C-ABI layer of the operators whose rows
// choose their weights (w8_grouped_api.cu) hands to their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "w8_grouped.h"
#include "w8_layout.h"
#include "w8_serve_internal.h"

namespace w8 {

struct RouteArgs {
    const void *x;
    int64_t ld;
    int toks, experts;
    const float *bias;
    int top, sigmoid, normalize;
    float scale;
    int32_t *ids;
    float *weights;
};
cudaError_t launch_route(const RouteArgs &a, bool bf16, cudaStream_t s);

// Items of one chunk are ranked by one CTA; up to kGroupOne items take one
// chunk and one launch, more at most kGroupChunks.  One chunk / chunks of 1024, us
// replayed, 64 groups: 1024 items 4.5 / 4.5 (one chunk either way), 2048 6.9 / 7.7,
// 4096 10.7 / 7.9, 8192 18.2 / 8.0, 16384 32.5 / 8.2 (256 groups a tenth more).  So
// chunks are the faster from about 2500 items on; up to 8192 are one chunk because
// those calls need no workspace, which is what callers are told.
constexpr int kGroupOne = 8192;
constexpr int kGroupChunks = 128;
struct GroupArgs {
    const int32_t *ids;
    int n, groups, per;
    int32_t *order, *rows, *offsets;
    int chunk, chunks;
    int32_t *counts; // [chunks][groups]
};
cudaError_t launch_group_rows(const GroupArgs &a, cudaStream_t s);

struct SumArgs {
    const uint16_t *y, *add;
    uint16_t *out;
    int64_t ldy, ld_add, ld_out;
    const int32_t *ids;
    const float *weights;
    int toks, top, n;
};
cudaError_t launch_expert_sum(const SumArgs &a, cudaStream_t s);

// The groups' planes: the first one's packed weights and row scales, and the
// distance from one group's to the next's.
struct GroupedArgs {
    w8_grouped a;
    const uint8_t *wp;
    const float *scale;
    int64_t wp_step, scale_step; // bytes, floats
    int n, k, kb, rt;
    int act;    // kActPlain, kActGateUp or kActSiluMul (w8_internal.h)
    int half;
    bool wide_y; // two columns of y may be stored together: 4-byte aligned, ldy even
};
cudaError_t launch_grouped(const GroupedArgs &a, bool fp8, int sms, cudaStream_t s);
cudaError_t grouped_status(int *out, bool reset);

int lora_splits(int n_rows, int k, int n_adapters, int sms);
size_t lora_ws_bytes(int n_rows, int rank, int sms);
cudaError_t lora_status(int *out, bool reset);
cudaError_t launch_lora(const w8_lora &a, float *v, int sms, cudaStream_t s);

} // namespace w8
