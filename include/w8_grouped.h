/*
 * w8_grouped.h -- C ABI of libw8, third part: the operators whose rows choose
 * their weights, for one GB300 GPU (sm_103a) -- the routed experts of a
 * mixture and the low-rank adapters of many requests, beside the projections
 * of w8.h.
 *
 *   w8_expert_route  router logits -> the chosen experts of each token and
 *                    their weights
 *   w8_group_rows    the chosen group of each row -> the rows in the order of
 *                    their groups, and where each group begins
 *   w8_grouped_gemv  each group's rows times that group's plane of a build
 *                    (plain, or gate_up with SiLU-and-multiply)
 *   w8_expert_sum    a token's expert outputs, weighted and added
 *   w8_lora_add      y += s_a B_a (A_a x), every row with its own adapter
 *
 * The conventions are those of w8.h and w8_serve.h: "device" pointers belong
 * to the current device, the caller owns every buffer, every function returns
 * a w8_status, arguments are checked on the host before anything is enqueued,
 * every call is asynchronous on the caller's stream and may be captured in a
 * CUDA graph (the first call of an operator on a device, of any size and type,
 * must come before a capture: it raises the shared-memory limits of all of the
 * operator's kernels).  Kernels are launched
 * with programmatic dependent launch and read no caller's buffer before the
 * previous kernel of the stream has completed.  No output may lie on an input,
 * but for out on y (or add), row on row, where a function says so.
 *
 * Values on the device (ids, offsets, row numbers) cannot be checked on the
 * host.  The kernels clamp or skip them so that no access leaves the buffers
 * that the arguments describe; what each does with a value out of range is
 * stated with the function.
 */
#ifndef W8_GROUPED_H
#define W8_GROUPED_H

#include "w8.h"
#include "w8_serve.h" /* W8_LOGITS_BF16, W8_LOGITS_F32 */

#ifdef __cplusplus
extern "C" {
#endif

#define W8_GROUPED_ABI_VERSION 1

/* Limits. */
#define W8_MAX_GROUPS 1024  /* experts of a router, groups, adapters of one call */
#define W8_MAX_ROUTED 32    /* experts of one token */
#define W8_MAX_RANK 128     /* of an adapter */

/* W8_GROUPED_ABI_VERSION of the loaded library. */
int w8_grouped_abi_version(void);

/* What a status code means for the functions of this header (static storage;
 * never NULL). */
const char *w8_grouped_status_str(w8_status s);

/* The status word of the tensor-memory kernels on the current device: 0 when
 * every bounded wait of every launch so far ended normally; otherwise bit 0
 * (w8_grouped_gemv) or bit 1 (w8_lora_add) is set and the outputs of some
 * launch are wrong.  Synchronous: it waits for all work of the device,
 * whatever its stream; reset != 0 clears the word. */
w8_status w8_grouped_device_status(int *status, int reset);

/* ---------------------------------------------------------------------------
 * The router.  For each token t, with x its n_experts logits:
 *   p_e = exp(x_e) / sum_f exp(x_f), or with `sigmoid` 1 / (1 + exp(-x_e));
 *   c_e = x_e, or with a bias (sigmoid only) p_e + bias_e;
 *   ids[t][0..top-1] = the experts of the `top` largest c_e, in falling order,
 *     the lowest number first among equal ones;
 *   weights[t][j] = scale * p of ids[t][j], with `normalize` divided by the
 *     sum of the chosen p.
 * The order is that of c_e in 64 bits: where fp32 cannot tell two of them apart
 * they are computed again (those that 64 bits cannot tell apart are equal).
 * Weights are fp32 throughout.
 * An expert whose logit (or bias) is -inf or NaN is never chosen and adds
 * nothing; a token with fewer than `top` experts left gets id -1 and weight 0
 * in the remaining places.  A logit of +inf gives NaN weights with softmax.
 * logits: device, dtype W8_LOGITS_BF16 (2-byte aligned) or W8_LOGITS_F32
 * (4-byte aligned), any ld >= n_experts; bias: device fp32 [n_experts], or
 * NULL; ids: device int32, weights: device fp32, [n_tok][top].
 * 1 <= n_experts <= W8_MAX_GROUPS, 1 <= top <= min(W8_MAX_ROUTED, n_experts);
 * scale: finite (W8_ERR_SCALE).  W8_ERR_LAYOUT: a bias without sigmoid.
 * n_tok = 0 is a no-op.  One kernel launch. */
w8_status w8_expert_route(const void *logits, int dtype, int64_t ld, int n_tok, int n_experts,
                          const float *bias, int top, int sigmoid, int normalize, float scale,
                          int32_t *ids, float *weights, w8_stream s);

/* ---------------------------------------------------------------------------
 * Rows by their groups.  ids[i] is the group of item i (0 .. n_groups - 1; any
 * other value: of none).  With items of one group in rising order:
 *   offsets[g] = items of groups before g, offsets[n_groups] = items of any;
 *   order[j], offsets[g] <= j < offsets[g + 1]: the items of group g;
 *   rows[j] = order[j] / per (the token of a routed pair; NULL: left out).
 * order[j] and rows[j] behind the last group's items are -1.
 * ids, order, rows: device int32 [n]; offsets: device int32 [n_groups + 1].
 * 0 <= n <= 2^30, 1 <= n_groups <= W8_MAX_GROUPS, per >= 1.  n = 0 sets the
 * offsets to 0.
 * workspace: w8_group_rows_workspace_bytes bytes (0 for few items: NULL then
 * does), 256-byte aligned; needs no initialisation; calls that share one must
 * not overlap on the GPU.  One kernel launch, two for many items. */
w8_status w8_group_rows(const int32_t *ids, int n, int n_groups, int per, int32_t *order, int32_t *rows,
                        int32_t *offsets, void *workspace, size_t workspace_bytes, w8_stream s);

/* Workspace bytes that serve every call of up to n items and n_groups groups
 * (host-only). */
w8_status w8_group_rows_workspace_bytes(int n, int n_groups, size_t *bytes);

/* ---------------------------------------------------------------------------
 * The groups' products.  Group g has positions offsets[g] .. offsets[g + 1]-1
 * and plane first + g * step of the build.  For each position i of group g:
 *   y[y_rows[i]][n] = bf16( scale_g[n] sum_k W_g[n][k] x[x_rows[i]][k] ),
 * without the scale on a bf16 build, or with silu_mul (planes bound as
 * W8_SRC_GATE_UP, n = 2I) for j < I
 *   y[y_rows[i]][j] = bf16( silu(g_j) u_j ),  silu(v) = v / (1 + exp(-v)),
 * g_j and u_j the scaled fp32 sums of source rows j and I + j.  Sums are fp32;
 * the one rounding is the output's (w8_gemv_silu_mul rounds g and u to bf16
 * first, as two steps would; here nothing reads them); silu(g) u is made within
 * 2^-19 of its value, for gates far below 0, too.  Without silu_mul a
 * gate_up plane's outputs are in source row order.
 * x: device bf16 [n_x][ldx], 16-byte aligned, ldx >= K and a multiple of 8;
 * y: device bf16 [n_y][ldy], 2-byte aligned; x_rows, y_rows: device int32
 * [n_rows], NULL for i itself; offsets: device int32 [n_groups + 1], cut to
 * 0 .. n_rows and taken as not decreasing.  A position whose row
 * of x is outside 0 .. n_x - 1 gives zeros, one whose row of y is outside
 * 0 .. n_y - 1 is not written; two positions with one row of y leave either's
 * values.  Rows of y that no position names are not written.  A NaN or infinity
 * in a row of x stays in that row's output.
 * The planes first, first + step, .. (n_groups of them) have one shape and
 * layout and lie at equal distances, as planes of a shape bound in turn do
 * (W8_ERR_LAYOUT otherwise, or with silu_mul on other planes); builds of
 * W8_DT_E4M3FN and W8_DT_BF16 (W8_ERR_DTYPE).  n_rows = 0 is a no-op.
 * One kernel launch, no workspace. */
typedef struct {
    const uint16_t *x;
    int64_t ldx;
    const int32_t *x_rows;
    uint16_t *y;
    int64_t ldy;
    const int32_t *y_rows;
    const int32_t *offsets;
    int32_t n_x, n_y;
    int32_t n_rows;
    int32_t first, step;     /* planes of the groups */
    int32_t n_groups;        /* 1 .. W8_MAX_GROUPS */
    int32_t silu_mul;
} w8_grouped;

w8_status w8_grouped_gemv(const w8_build *b, const w8_grouped *a, w8_stream s);

/* ---------------------------------------------------------------------------
 * out[t][c] = bf16( add[t][c] + sum_j weights[t][j] y[t * top + j][c] ), over
 * the j with ids[t][j] >= 0, in rising order of j, in fp32 (rows of y of the
 * others are not read; ids NULL: all count; add NULL: 0).
 * y: device bf16 [n_tok * top][ldy]; ids: device int32, weights: device fp32
 * [n_tok][top]; add, out: device bf16 [n_tok][ld..]; all 2-byte aligned (16
 * bytes and strides in multiples of 8 are faster); out may be add.
 * 1 <= top <= W8_MAX_ROUTED, 1 <= n <= 2^22.  n_tok = 0 is a no-op.  One
 * kernel launch. */
w8_status w8_expert_sum(const uint16_t *y, int64_t ldy, const int32_t *ids, const float *weights,
                        const uint16_t *add, int64_t ld_add, uint16_t *out, int64_t ld_out, int n_tok,
                        int top, int n, w8_stream s);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection.  Adapter a
 * has positions offsets[a] .. offsets[a + 1] - 1 of order, each naming a row t
 * of x, y and out:
 *   v = A_a x[t]  (rank_a sums over k, fp32)
 *   out[t][c] = bf16( y[t][c] + scales[a] sum_j B_a[c][j] v_j ),  c < n.
 * v enters the second product as the sum of two bf16 values, so that nothing
 * of it is lost above 2^-16 (an infinity in B may give NaN: one of the two may
 * be 0); all sums are fp32.  Rows that no position names
 * are not written; a row outside 0 .. n_tok - 1 is skipped.  Of two positions
 * with one row either's result is left (with out on y perhaps both added): a
 * token has one adapter.
 * x: device bf16 [n_tok][ldx]; a: device bf16 [n_adapters][rank][k], adapters
 * ld_a apart, rows ld_a_row; b: device bf16 [n_adapters][n][rank], adapters
 * ld_b apart, rows ld_b_row; all three 16-byte aligned with strides in
 * multiples of 8.  y, out: device bf16 [n_tok][ldy, ld_out], 2-byte aligned
 * (16 bytes and strides in multiples of 8 are faster); out may be y.  order:
 * device int32 [n_rows]; offsets: device int32 [n_adapters + 1], cut to
 * 0 .. n_rows and taken as not decreasing; ranks: device int32 [n_adapters],
 * cut to 0 .. rank, NULL for rank (what A and B hold past an adapter's rank is
 * not used, nor what B's rows hold past it); scales: device fp32
 * [n_adapters], NULL for 1.
 * 1 <= rank <= W8_MAX_RANK, 1 <= n_adapters <= W8_MAX_GROUPS, k and n up to
 * 2^23.  n_rows = 0 is a no-op.
 * workspace: w8_lora_workspace_bytes bytes, 256-byte aligned; needs no
 * initialisation; calls that share one must not overlap on the GPU.  Two
 * kernel launches. */
typedef struct {
    const uint16_t *x;
    int64_t ldx;
    const uint16_t *a;
    int64_t ld_a, ld_a_row;
    const uint16_t *b;
    int64_t ld_b, ld_b_row;
    const uint16_t *y;
    int64_t ldy;
    uint16_t *out;
    int64_t ld_out;
    const int32_t *order;
    const int32_t *offsets;
    const int32_t *ranks;
    const float *scales;
    int32_t n_tok, n_rows;
    int32_t n_adapters;
    int32_t k, n, rank;
} w8_lora;

w8_status w8_lora_add(const w8_lora *a, void *workspace, size_t workspace_bytes, w8_stream s);

/* Workspace bytes that serve every call of up to n_rows positions, k columns,
 * this rank or less and n_adapters adapters on a GPU of sm_count SMs
 * (host-only). */
w8_status w8_lora_workspace_bytes(int n_rows, int k, int rank, int n_adapters, int sm_count, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* W8_GROUPED_H */
