// w8_serve_api.cu -- the C ABI of the serving operators (declared and
// documented in include/w8_serve.h): host-side checks, then one launch call.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "w8_serve.h"
#include "w8_serve_internal.h"

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 38; // elements; tensor-map strides stay below 2^40 bytes
constexpr int64_t kMaxItems = int64_t(1) << 30; // rows of an output, tokens, logits of a row

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A bf16 operand read with 16-byte loads or tensor-map copies: 16-byte
// aligned, strides of at least `least` elements and multiples of 8.
w8_status check_vec(const void *p, int64_t ld_tok, int64_t least_tok, int64_t ld_head, int64_t least_head)
{
    if (!p)
        return W8_ERR_NULL;
    if (ld_tok < least_tok || ld_head < least_head || ld_tok > kMaxStride || ld_head > kMaxStride)
        return W8_ERR_SHAPE;
    return aligned(p, 16) && ld_tok % 8 == 0 && ld_head % 8 == 0 ? W8_OK : W8_ERR_ALIGN;
}

w8_status check_cache(const w8_latent_cache &c)
{
    if (!c.data)
        return W8_ERR_NULL;
    if (c.n_pages < 1 || c.page_size < 1 || c.page_size > (1 << 20) || c.ld_tok < W8_LATENT_ROW ||
        c.ld_tok > kMaxStride || c.ld_page > kMaxStride ||
        c.ld_page < int64_t(c.page_size - 1) * c.ld_tok + W8_LATENT_ROW)
        return W8_ERR_SHAPE;
    return aligned(c.data, 16) && c.ld_tok % 8 == 0 && c.ld_page % 8 == 0 ? W8_OK : W8_ERR_ALIGN;
}

struct Range {
    const void *p;
    int64_t bytes;
};
// Whether a range meets one of `rows` rows of `bytes` bytes, `ld` bytes apart.
bool meets(const Range &a, const void *p, int64_t rows, int64_t ld, int64_t bytes)
{
    if (a.bytes <= 0 || bytes <= 0)
        return false;
    const int64_t at = int64_t(reinterpret_cast<uintptr_t>(a.p)) - int64_t(reinterpret_cast<uintptr_t>(p)); // from the first row
    const int64_t row = at < bytes ? 0 : (at - bytes) / ld + 1; // the first row that ends behind the range's start
    return row < rows && row * ld < at + a.bytes;
}

// SMs of the current device; 0 on failure.
int current_sms()
{
    int dev = -1, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

w8_status launched(cudaError_t e) { return e == cudaSuccess ? W8_OK : W8_ERR_CUDA; }

#define W8_TRY(expr)                    \
    do {                                \
        const w8_status st_ = (expr);   \
        if (st_ != W8_OK)               \
            return st_;                 \
    } while (0)

} // namespace

extern "C" {

int w8_serve_abi_version(void) { return W8_SERVE_ABI_VERSION; }

const char *w8_serve_status_str(w8_status s)
{
    switch (s) {
    case W8_OK: return "ok";
    case W8_ERR_NULL: return "a required pointer is NULL";
    case W8_ERR_DTYPE: return "logits are bf16 or fp32";
    case W8_ERR_SHAPE: return "a count, stride or head shape outside what the function takes "
                              "(limits: w8_serve.h), or an output of w8_block_tables on one of "
                              "its inputs";
    case W8_ERR_SCALE: return "the softmax scale must be finite and above zero";
    case W8_ERR_CAPACITY: return "workspace too small";
    case W8_ERR_ALIGN: return "misaligned operand (bf16 operands: 16 B with strides in multiples "
                              "of 8; workspace: 256 B)";
    case W8_ERR_CUDA: return "CUDA runtime error";
    default: return w8_status_str(s);
    }
}

w8_status w8_serve_device_status(int *status, int reset)
{
    if (!status)
        return W8_ERR_NULL;
    // all streams' launches so far: the copies below wait for none that does not block
    if (cudaDeviceSynchronize() != cudaSuccess)
        return W8_ERR_CUDA;
    int paged = 0, expanded = 0, pairs = 0;
    if (w8::paged_status(&paged, reset != 0) != cudaSuccess || w8::expanded_status(&expanded, reset != 0) != cudaSuccess ||
        w8::pairs_status(&pairs, reset != 0) != cudaSuccess)
        return W8_ERR_CUDA;
    *status = (paged ? 1 : 0) | (expanded || pairs ? 2 : 0);
    return W8_OK;
}

w8_status w8_block_tables(const int32_t *ctx_lens, const int32_t *new_lens, int n_req, int page_size,
                          const int32_t *free_pages, int n_free, const int32_t *free_head,
                          int32_t *block_table, int64_t ld_table, int max_pages,
                          int32_t *seq_lens, int32_t *cu_new, int64_t *slots, int32_t *positions,
                          int max_tokens, int32_t *free_head_out, int32_t *status, w8_stream s)
{
    if (n_req < 1 || n_req > W8_MAX_REQUESTS || page_size < 1 || page_size > (1 << 20) || n_free < 0 ||
        max_pages < 1 || ld_table < max_pages || ld_table > kMaxStride || max_tokens < 0 ||
        max_tokens > kMaxItems)
        return W8_ERR_SHAPE;
    if (!ctx_lens || !new_lens || (n_free > 0 && !free_pages) || !free_head || !block_table || !seq_lens ||
        !cu_new || (max_tokens > 0 && (!slots || !positions)) || !free_head_out || !status)
        return W8_ERR_NULL;
    if (free_head == free_head_out)
        return W8_ERR_SHAPE;
    if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) || !aligned(free_head, 4) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_new, 4) || !aligned(slots, 8) ||
        !aligned(positions, 4) || !aligned(free_head_out, 4) || !aligned(status, 4))
        return W8_ERR_ALIGN;
    // Every CTA reads all lengths while others write: no output may lie on an input.
    const int64_t n = n_req, toks = max_tokens;
    const Range in[] = {{ctx_lens, 4 * n}, {new_lens, 4 * n}, {free_pages, 4 * int64_t(n_free)}, {free_head, 4}},
                out[] = {{seq_lens, 4 * n},  {cu_new, 4 * (n + 1)}, {slots, 8 * toks},
                         {positions, 4 * toks}, {free_head_out, 4},    {status, 4}};
    for (const Range &i : in) {
        for (const Range &o : out)
            if (meets(i, o.p, 1, 1, o.bytes))
                return W8_ERR_SHAPE;
        if (meets(i, block_table, n, 4 * ld_table, 4 * int64_t(max_pages)))
            return W8_ERR_SHAPE;
    }
    const int sms = current_sms();
    if (sms < 1)
        return W8_ERR_CUDA;
    w8::TableArgs a{};
    a.ctx = ctx_lens;
    a.fresh = new_lens;
    a.free_pages = free_pages;
    a.free_head = free_head;
    a.table = block_table;
    a.seq_lens = seq_lens;
    a.cu = cu_new;
    a.positions = positions;
    a.head_out = free_head_out;
    a.status = status;
    a.slots = slots;
    a.ld_table = ld_table;
    a.n_req = n_req;
    a.page = page_size;
    a.n_free = n_free;
    a.max_pages = max_pages;
    a.max_tok = max_tokens;
    return launched(w8::launch_block_tables(a, sms, reinterpret_cast<cudaStream_t>(s)));
}

w8_status w8_latent_cache_write(const uint16_t *latent, int64_t ld_latent, const uint16_t *rope,
                                int64_t ld_rope, const int64_t *slots, int n_tok,
                                const w8_latent_cache *cache, w8_stream s)
{
    if (n_tok < 0 || n_tok > kMaxItems)
        return W8_ERR_SHAPE;
    if (n_tok == 0)
        return W8_OK;
    if (!cache || !slots)
        return W8_ERR_NULL;
    W8_TRY(check_cache(*cache));
    W8_TRY(check_vec(latent, ld_latent, W8_LATENT_DIM, 0, 0));
    W8_TRY(check_vec(rope, ld_rope, W8_LATENT_ROPE, 0, 0));
    if (!aligned(slots, 8))
        return W8_ERR_ALIGN;
    w8::CacheWriteArgs a{};
    a.latent = latent;
    a.rope = rope;
    a.ld_latent = ld_latent;
    a.ld_rope = ld_rope;
    a.slots = slots;
    a.cache = static_cast<uint16_t *>(cache->data);
    a.ld_page = cache->ld_page;
    a.ld_tok = cache->ld_tok;
    a.n_slots = int64_t(cache->n_pages) * cache->page_size;
    a.page = cache->page_size;
    a.n_tok = n_tok;
    return launched(w8::launch_cache_write(a, reinterpret_cast<cudaStream_t>(s)));
}

w8_status w8_latent_paged_workspace_bytes(int n_tok, int n_heads, int n_req, int sm_count, size_t *bytes)
{
    if (!bytes)
        return W8_ERR_NULL;
    if (n_tok < 0 || n_heads < 1 || n_heads > W8_MAX_LATENT_HEADS || n_req < 1 || n_req > W8_MAX_REQUESTS ||
        sm_count < 1 || int64_t(n_tok) * n_heads > kMaxItems)
        return W8_ERR_SHAPE;
    *bytes = w8::latent_paged_ws_bytes(n_tok, n_heads, n_req, sm_count);
    return W8_OK;
}

w8_status w8_latent_attn_paged(const w8_latent_paged *a, void *workspace, size_t workspace_bytes,
                               w8_stream s)
{
    if (!a)
        return W8_ERR_NULL;
    if (a->n_tok < 0 || a->n_heads < 1 || a->n_heads > W8_MAX_LATENT_HEADS || a->n_req < 1 ||
        a->n_req > W8_MAX_REQUESTS || int64_t(a->n_tok) * a->n_heads > kMaxItems || a->max_pages < 1 ||
        a->ld_table < a->max_pages || a->ld_table > kMaxStride)
        return W8_ERR_SHAPE;
    if (a->n_tok == 0)
        return W8_OK;
    if (!(a->scale > 0.0f) || !isfinite(a->scale))
        return W8_ERR_SCALE;
    W8_TRY(check_cache(a->cache));
    if (a->cache.page_size < 16 || a->cache.page_size > 1024 || (a->cache.page_size & (a->cache.page_size - 1)))
        return W8_ERR_SHAPE;
    W8_TRY(check_vec(a->q_lat, a->ld_qlat_tok, W8_LATENT_DIM, a->ld_qlat_head, W8_LATENT_DIM));
    W8_TRY(check_vec(a->q_rope, a->ld_qrope_tok, W8_LATENT_ROPE, a->ld_qrope_head, W8_LATENT_ROPE));
    if (!a->block_table || !a->seq_lens || !a->cu_q || !a->out)
        return W8_ERR_NULL;
    if (a->ld_out_tok < W8_LATENT_DIM || a->ld_out_head < W8_LATENT_DIM || a->ld_out_tok > kMaxStride ||
        a->ld_out_head > kMaxStride)
        return W8_ERR_SHAPE;
    if (!aligned(a->out, 4) || a->ld_out_tok % 2 || a->ld_out_head % 2 || !aligned(a->lse, 4) ||
        !aligned(a->block_table, 4) || !aligned(a->seq_lens, 4) || !aligned(a->cu_q, 4))
        return W8_ERR_ALIGN;
    const int sms = current_sms();
    if (sms < 1)
        return W8_ERR_CUDA;
    const size_t need = w8::latent_paged_ws_bytes(a->n_tok, a->n_heads, a->n_req, sms);
    if (need > 0 && !workspace)
        return W8_ERR_NULL;
    if (!aligned(workspace, 256))
        return W8_ERR_ALIGN;
    if (workspace_bytes < need)
        return W8_ERR_CAPACITY;
    return launched(w8::launch_latent_paged(*a, workspace, sms, reinterpret_cast<cudaStream_t>(s)));
}

w8_status w8_latent_attn_expanded(const w8_latent_expanded *a, w8_stream s)
{
    if (!a)
        return W8_ERR_NULL;
    if (!((a->d_nope == 192 && a->d_v == 256) || (a->d_nope == 128 && a->d_v == 128)) || a->n_q < 0 ||
        a->n_k < 0 || a->n_k > kMaxItems || a->n_heads < 1 || a->n_heads > W8_MAX_LATENT_HEADS || a->n_req < 1 ||
        a->n_req > W8_MAX_REQUESTS || int64_t(a->n_q) * a->n_heads > kMaxItems)
        return W8_ERR_SHAPE;
    if (a->n_q == 0)
        return W8_OK;
    if (!(a->scale > 0.0f) || !isfinite(a->scale))
        return W8_ERR_SCALE;
    W8_TRY(check_vec(a->q_nope, a->ld_qnope_tok, a->d_nope, a->ld_qnope_head, a->d_nope));
    W8_TRY(check_vec(a->q_rope, a->ld_qrope_tok, W8_LATENT_ROPE, a->ld_qrope_head, W8_LATENT_ROPE));
    if (a->n_k > 0) {
        W8_TRY(check_vec(a->k_nope, a->ld_knope_tok, a->d_nope, a->ld_knope_head, a->d_nope));
        W8_TRY(check_vec(a->k_rope, a->ld_krope_tok, W8_LATENT_ROPE, 0, 0));
        W8_TRY(check_vec(a->v, a->ld_v_tok, a->d_v, a->ld_v_head, a->d_v));
    }
    W8_TRY(check_vec(a->out, a->ld_out_tok, a->d_v, a->ld_out_head, a->d_v));
    if (!a->cu_q || !a->cu_k)
        return W8_ERR_NULL;
    if (!aligned(a->lse, 4) || !aligned(a->cu_q, 4) || !aligned(a->cu_k, 4))
        return W8_ERR_ALIGN;
    const int sms = current_sms();
    if (sms < 1)
        return W8_ERR_CUDA;
    return launched(w8::launch_latent_expanded(*a, sms, reinterpret_cast<cudaStream_t>(s)));
}

static size_t logprobs_ws_bytes(int n_rows, int vocab, int sms)
{
    const int splits = w8::logprobs_splits(n_rows, vocab, sms);
    return splits < 2 ? 0
                      : w8::kLogprobsCounters * sizeof(int) +
                            size_t(n_rows) * size_t(splits) * sizeof(w8::LogprobsPart);
}

w8_status w8_logprobs_workspace_bytes(int n_rows, int vocab, int top, int sm_count, size_t *bytes)
{
    if (!bytes)
        return W8_ERR_NULL;
    if (n_rows < 0 || n_rows > kMaxItems || vocab < 1 || vocab > kMaxItems || top < 0 || top > W8_MAX_TOP ||
        top > vocab || sm_count < 1)
        return W8_ERR_SHAPE;
    *bytes = n_rows == 0 ? 0 : logprobs_ws_bytes(n_rows, vocab, sm_count);
    return W8_OK;
}

w8_status w8_logprobs_workspace_bytes_upto(int n_rows, int vocab, int top, int sm_count, size_t *bytes)
{
    size_t most = 0;
    const w8_status st = w8_logprobs_workspace_bytes(n_rows, vocab, top, sm_count, bytes);
    if (st != W8_OK)
        return st;
    // Fewer rows are cut into more runs each, and may need more than many that are
    // not cut; a smaller vocabulary never needs more.
    for (int rows = 1; rows <= n_rows; ++rows) {
        const size_t need = logprobs_ws_bytes(rows, vocab, sm_count);
        if (need == 0) // nor do more rows
            break;
        most = need > most ? need : most;
    }
    *bytes = most;
    return W8_OK;
}

w8_status w8_token_logprobs(const void *logits, int dtype, int64_t ld, int n_rows, int vocab,
                            const int32_t *tokens, float *logprob, float *entropy, int top,
                            int32_t *top_ids, float *top_logprobs, void *workspace,
                            size_t workspace_bytes, w8_stream s)
{
    if (dtype != W8_LOGITS_BF16 && dtype != W8_LOGITS_F32)
        return W8_ERR_DTYPE;
    if (n_rows < 0 || n_rows > kMaxItems || vocab < 1 || vocab > kMaxItems || ld < vocab || ld > kMaxStride ||
        top < 0 || top > W8_MAX_TOP || top > vocab)
        return W8_ERR_SHAPE;
    if (n_rows == 0)
        return W8_OK;
    if (!logits || !tokens || !logprob || (top > 0 && (!top_ids || !top_logprobs)))
        return W8_ERR_NULL;
    if (!aligned(logits, dtype == W8_LOGITS_BF16 ? 2 : 4) || !aligned(tokens, 4) || !aligned(logprob, 4) ||
        !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
        return W8_ERR_ALIGN;
    const int sms = current_sms();
    if (sms < 1)
        return W8_ERR_CUDA;
    const size_t need = logprobs_ws_bytes(n_rows, vocab, sms);
    if (need > 0 && !workspace)
        return W8_ERR_NULL;
    if (need > 0 && !aligned(workspace, 256))
        return W8_ERR_ALIGN;
    if (workspace_bytes < need)
        return W8_ERR_CAPACITY;
    w8::LogprobsArgs a{};
    a.x = logits;
    a.ld = ld;
    a.rows = n_rows;
    a.vocab = vocab;
    a.top = top;
    a.splits = w8::logprobs_splits(n_rows, vocab, sms);
    a.tokens = tokens;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.counters = static_cast<int *>(workspace);
    a.parts = reinterpret_cast<w8::LogprobsPart *>(static_cast<uint8_t *>(workspace) +
                                                   w8::kLogprobsCounters * sizeof(int));
    return launched(w8::launch_logprobs(a, dtype == W8_LOGITS_BF16, reinterpret_cast<cudaStream_t>(s)));
}

} // extern "C"
