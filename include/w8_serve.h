/*
 * w8_serve.h -- C ABI of libw8, second part: the operators that a decode or
 * prefill step runs between and after the projections of w8.h, for one GB300
 * GPU (sm_103a).
 *
 *   w8_block_tables         lengths of the requests -> pages, block tables,
 *                           sequence lengths, query offsets, slot map
 *   w8_latent_cache_write   latent and rope-key rows -> their slots of a
 *                           paged cache
 *   w8_latent_attn_paged    latent attention, absorbed form: queries already
 *                           carried into the latent space, over the paged
 *                           cache (decode and draft rows)
 *   w8_latent_attn_expanded latent attention, expanded form: keys and values
 *                           as the kv_b projection writes them (prompts)
 *   w8_token_logprobs       logits -> log probability of a given token,
 *                           entropy, most likely alternatives
 *
 * The conventions are those of w8.h: "device" pointers belong to the current
 * device, the caller owns every buffer, every function returns a w8_status,
 * arguments are checked on the host before anything is enqueued, every call
 * is asynchronous on the caller's stream and may be captured in a CUDA graph
 * (the first call of an operator on a device must come before a capture: it
 * raises the kernels' shared-memory limits).  Kernels are launched with
 * programmatic dependent launch and touch no global memory before the
 * previous kernel of the stream has completed.
 *
 * Values on the device (lengths, offsets, page numbers) cannot be checked on
 * the host.  The kernels clamp them so that no access leaves the buffers that
 * the arguments describe; what each does with a value out of range is stated
 * with the function.
 */
#ifndef W8_SERVE_H
#define W8_SERVE_H

#include "w8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define W8_SERVE_ABI_VERSION 2

/* Columns of a latent-cache row: the latent, then the rope key shared by all
 * heads (kv_a_proj_with_mqa's 576 rows). */
#define W8_LATENT_DIM 512
#define W8_LATENT_ROPE 64
#define W8_LATENT_ROW (W8_LATENT_DIM + W8_LATENT_ROPE)

/* Limits. */
#define W8_MAX_REQUESTS 16384  /* requests of one call */
#define W8_MAX_LATENT_HEADS 256
#define W8_MAX_TOP 32          /* alternatives of w8_token_logprobs */

/* W8_SERVE_ABI_VERSION of the loaded library. */
int w8_serve_abi_version(void);

/* What a status code means for the functions of this header (static storage;
 * never NULL). */
const char *w8_serve_status_str(w8_status s);

/* The status word of the attention kernels on the current device: 0 when every
 * bounded wait of every launch so far ended normally; otherwise bit 0 (paged
 * form) or bit 1 (expanded form) is set and the outputs of some launch are
 * wrong.  Synchronous: it waits for all work of the device, whatever its
 * stream; reset != 0 clears the word. */
w8_status w8_serve_device_status(int *status, int reset);

/* ---------------------------------------------------------------------------
 * Paged bookkeeping of one step, on the GPU.  Request r holds ctx_lens[r]
 * tokens in the cache and appends new_lens[r]; pages hold page_size tokens.
 * With have_r = ceil(ctx / page_size), want_r = ceil((ctx + new) / page_size),
 * both cut at max_pages, and base_r = *free_head + sum_{r' < r} (want - have):
 *   block_table[r][p] = free_pages[base_r + p - have_r],  have_r <= p < want_r
 *   seq_lens[r] = ctx + new,   cu_new[r] = sum_{r' < r} new,  cu_new[n_req] = all
 *   (the sums cut at 2^31 - 1)
 *   for token t of request r, pos = ctx_r + t - cu_new[r]:
 *     positions[t] = pos,
 *     slots[t] = block_table[r][pos / page_size] * page_size + pos % page_size
 *   *free_head_out = *free_head + sum (want - have), at most n_free.
 * Entries of a table row outside [have, want) are neither read (except the
 * page that a partly filled tail continues) nor written.  slots and positions
 * past the last token, up to max_tokens, are -1 (the padding rows of a
 * captured step).
 * *status (device) is 0, or the sum of
 *   1: the free list ran out: the missing entries are -1, and so are the
 *      slots of their tokens;
 *   2: a request outgrew its table row: its tokens past max_pages * page_size
 *      have slot -1, and no page is taken for them;
 *   4: a length below zero (taken as 0), a sequence past 2^31 - 1 tokens (cut
 *      there), or more than max_tokens tokens (those past it get no slot).
 * ctx_lens, new_lens: device int32 [n_req]; free_pages: device int32
 * [n_free]; free_head, free_head_out: device int32; block_table: device int32
 * [n_req][ld_table], ld_table >= max_pages; seq_lens [n_req], cu_new
 * [n_req + 1], positions [max_tokens]: device int32; slots: device int64
 * [max_tokens]; status: device int32.  No output may lie on an input (lengths
 * are not advanced in place, a step that is run again gives the same answer):
 * W8_ERR_SHAPE.
 * 1 <= n_req <= W8_MAX_REQUESTS, max_pages >= 1, max_tokens >= 0,
 * 1 <= page_size <= 2^20.  One kernel launch. */
w8_status w8_block_tables(const int32_t *ctx_lens, const int32_t *new_lens, int n_req, int page_size,
                          const int32_t *free_pages, int n_free, const int32_t *free_head,
                          int32_t *block_table, int64_t ld_table, int max_pages,
                          int32_t *seq_lens, int32_t *cu_new, int64_t *slots, int32_t *positions,
                          int max_tokens, int32_t *free_head_out, int32_t *status, w8_stream s);

/* A paged latent cache: bf16 [n_pages][page_size][W8_LATENT_ROW], rows ld_tok
 * elements apart, pages ld_page elements apart; 16-byte aligned, both strides
 * multiples of 8.  Token j of a request is row j % page_size of page
 * block_table[j / page_size]. */
typedef struct {
    void *data;        /* device */
    int64_t ld_page;   /* >= (page_size - 1) * ld_tok + W8_LATENT_ROW */
    int64_t ld_tok;    /* >= W8_LATENT_ROW */
    int32_t n_pages;   /* >= 1 */
    int32_t page_size; /* w8_latent_attn_paged: a power of two, 16 .. 1024 */
} w8_latent_cache;

/* cache row slots[t] = [latent[t][0..511] | rope[t][0..63]], t < n_tok.  A
 * slot outside [0, n_pages * page_size) is skipped; two tokens with one slot
 * leave either's row (per 16 bytes).
 * latent, rope: device bf16, 16-byte aligned, row strides multiples of 8
 * (slices of the merged qkv_a output fit); slots: device int64 [n_tok].
 * n_tok = 0 is a no-op.  One kernel launch. */
w8_status w8_latent_cache_write(const uint16_t *latent, int64_t ld_latent, const uint16_t *rope,
                                int64_t ld_rope, const int64_t *slots, int n_tok,
                                const w8_latent_cache *cache, w8_stream s);

/* ---------------------------------------------------------------------------
 * Latent attention, absorbed form.  Request r has query tokens
 * cu_q[r] .. cu_q[r+1]-1, the last of its seq_lens[r] cached tokens (their
 * own rows are in the cache already).  For query token i of the request (of
 * n = cu_q[r+1] - cu_q[r]) and head h, over cached tokens
 * j <= seq_lens[r] - n + i, with c_j the latent and e_j the rope key:
 *   x_j = scale * (q_lat[t][h] . c_j + q_rope[t][h] . e_j)
 *   lse[t][h] = ln sum_j exp(x_j),   out[t][h] = sum_j exp(x_j - lse) c_j.
 * A query that sees nothing gives out 0 and lse -inf.  Scores, the softmax
 * and both sums are fp32; the weights are rounded to bf16 for the second
 * product (the sum that divides them is of the unrounded ones), out is
 * rounded to bf16 once.
 * q_lat: device bf16 [n_tok][n_heads][512]; q_rope [n_tok][n_heads][64]; both
 * 16-byte aligned with token and head strides multiples of 8.  out: device
 * bf16, 4-byte aligned, token and head strides multiples of 2; lse: device
 * fp32 [n_tok][n_heads], or NULL.
 * seq_lens [n_req], cu_q [n_req + 1], block_table [n_req][ld_table]: device
 * int32.  cu_q must not decrease; it is cut to 0 .. n_tok, seq_lens to
 * 0 .. max_pages * page_size.  Tokens that no request holds are not written.
 * Cached rows past a request's length are never used, whatever they hold; a
 * page number outside the cache reads as zeros.  A non-finite value in a
 * cached token reaches the query tokens that see it, and no other.
 * scale: finite, > 0.  n_tok = 0 is a no-op.
 * workspace: w8_latent_paged_workspace_bytes bytes, 256-byte aligned; needs
 * no initialisation; calls that share one must not overlap on the GPU.
 * Two kernel launches. */
typedef struct {
    const uint16_t *q_lat;
    int64_t ld_qlat_tok, ld_qlat_head;
    const uint16_t *q_rope;
    int64_t ld_qrope_tok, ld_qrope_head;
    w8_latent_cache cache;
    const int32_t *block_table;
    int64_t ld_table;       /* >= max_pages */
    const int32_t *seq_lens;
    const int32_t *cu_q;
    uint16_t *out;
    int64_t ld_out_tok, ld_out_head;
    float *lse;
    int32_t max_pages;      /* columns of block_table, >= 1 */
    int32_t n_req;          /* 1 .. W8_MAX_REQUESTS */
    int32_t n_tok;
    int32_t n_heads;        /* 1 .. W8_MAX_LATENT_HEADS */
    float scale;
} w8_latent_paged;

w8_status w8_latent_attn_paged(const w8_latent_paged *a, void *workspace, size_t workspace_bytes,
                               w8_stream s);

/* Workspace bytes of such a call on a GPU of sm_count SMs (host-only). */
w8_status w8_latent_paged_workspace_bytes(int n_tok, int n_heads, int n_req, int sm_count,
                                          size_t *bytes);

/* ---------------------------------------------------------------------------
 * Latent attention, expanded form.  Request r has query tokens cu_q[r] ..
 * cu_q[r+1]-1 (nq of them) and keys cu_k[r] .. cu_k[r+1]-1 (nk).  For query i
 * of the request and head h, over its keys j (causal: j <= nk - nq + i):
 *   x_j = scale * (q_nope[i][h] . k_nope[j][h] + q_rope[i][h] . k_rope[j])
 *   lse = ln sum_j exp(x_j),   out = sum_j exp(x_j - lse) v[j][h].
 * A query that sees nothing gives out 0 and lse -inf.  Precision as in the
 * paged form.  Head shapes (d_nope, rope, d_v): (192, 64, 256) and
 * (128, 64, 128).
 * All inputs device bf16, 16-byte aligned, strides multiples of 8: q_nope
 * [n_q][n_heads][d_nope], q_rope [n_q][n_heads][64], k_nope
 * [n_k][n_heads][d_nope], k_rope [n_k][64] (shared by the heads), v
 * [n_k][n_heads][d_v]; slices of the q_b and kv_b outputs fit.  out: device
 * bf16, 16-byte aligned, strides multiples of 8; lse: device fp32
 * [n_q][n_heads], or NULL.  cu_q, cu_k [n_req + 1]: device int32, not
 * decreasing; cut to 0 .. n_q and 0 .. n_k.  Keys of other requests are never
 * used, whatever they hold, nor are keys that causality hides from a query.
 * scale: finite, > 0.  n_q = 0 is a no-op; n_k may be 0.  One kernel launch. */
typedef struct {
    const uint16_t *q_nope;
    int64_t ld_qnope_tok, ld_qnope_head;
    const uint16_t *q_rope;
    int64_t ld_qrope_tok, ld_qrope_head;
    const uint16_t *k_nope;
    int64_t ld_knope_tok, ld_knope_head;
    const uint16_t *k_rope;
    int64_t ld_krope_tok;
    const uint16_t *v;
    int64_t ld_v_tok, ld_v_head;
    const int32_t *cu_q;
    const int32_t *cu_k;
    uint16_t *out;
    int64_t ld_out_tok, ld_out_head;
    float *lse;
    int32_t n_req;
    int32_t n_q;
    int32_t n_k;
    int32_t n_heads;        /* 1 .. W8_MAX_LATENT_HEADS */
    int32_t d_nope, d_v;
    int32_t causal;         /* 0: every query sees every key of its request */
    float scale;
} w8_latent_expanded;

w8_status w8_latent_attn_expanded(const w8_latent_expanded *a, w8_stream s);

/* ---------------------------------------------------------------------------
 * For each row i of logits [n_rows][ld] (vocab columns), with x its logits and
 * lse = ln sum_v exp(x_v):
 *   logprob[i] = x[tokens[i]] - lse
 *   entropy[i] = -sum_v p_v ln p_v,  p_v = exp(x_v - lse)   (NULL: left out)
 *   top_ids[i][0..top-1], top_logprobs[i][0..top-1]: the `top` largest logits
 *   in falling order, the lowest index first among equal ones, and their log
 *   probabilities x - lse.
 * Logits of -inf (banned tokens) have probability 0 and add nothing to the
 * entropy.  A row whose every logit is -inf, or that holds +inf or NaN, gives
 * NaN (0/0, inf - inf); its top_ids are then token numbers in no stated order
 * (all -inf: 0, 1, ...).  A token outside [0, vocab) reads nothing and gives
 * logprob NaN.  All sums are fp32.
 * logits: device, dtype W8_LOGITS_BF16 (2-byte aligned) or W8_LOGITS_F32
 * (4-byte aligned), any ld >= vocab; tokens: device int32 [n_rows]; logprob,
 * entropy: device fp32 [n_rows]; top_ids int32 and top_logprobs fp32
 * [n_rows][top], NULL when top is 0.  0 <= top <= min(W8_MAX_TOP, vocab).
 * n_rows = 0 is a no-op.
 * workspace: w8_logprobs_workspace_bytes bytes or more, 256-byte aligned,
 * zero-filled once before its first use; every call, whatever its shape, leaves
 * its counters at zero again; calls that share one must not overlap on the GPU.  One kernel launch. */
#define W8_LOGITS_BF16 1
#define W8_LOGITS_F32 2
w8_status w8_token_logprobs(const void *logits, int dtype, int64_t ld, int n_rows, int vocab,
                            const int32_t *tokens, float *logprob, float *entropy, int top,
                            int32_t *top_ids, float *top_logprobs, void *workspace,
                            size_t workspace_bytes, w8_stream s);

/* Workspace bytes of such a call on a GPU of sm_count SMs (host-only).  They do
 * not grow with the rows: many rows need none. */
w8_status w8_logprobs_workspace_bytes(int n_rows, int vocab, int top, int sm_count, size_t *bytes);

/* Workspace bytes that serve every call of up to n_rows rows, vocab columns and
 * top alternatives (host-only). */
w8_status w8_logprobs_workspace_bytes_upto(int n_rows, int vocab, int top, int sm_count, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* W8_SERVE_H */
