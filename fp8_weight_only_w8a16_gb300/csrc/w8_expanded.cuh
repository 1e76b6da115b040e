// w8_expanded.cuh -- what the two kernels of latent attention's expanded form
// share (w8_latent_expanded.cu: one CTA by itself; w8_latent_pair.cu: pairs of
// CTAs): the softmax of a tile, the tensor maps, the launch arguments.
//
// With s = scale log2 e and a running reference m_i of query i,
//   x_ij = q_i . k_j,  p_ij = 2^(s x_ij - m_i),  z_i = sum_j p_ij,
//   out_i = sum_j p_ij v_j / z_i,  lse_i = (m_i + log2 z_i) ln 2.
// A CTA holds 128 queries and walks over the keys they see, 128 at a time, with
// S [128 x 128] and O [128 x d_v] in tensor memory, a query a lane.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "w8_serve_internal.h"
#include "w8_tcgen.cuh"

namespace w8 {
namespace expanded {

using namespace tcg;

constexpr int kRows = 128, kKeys = 128;       // queries of a CTA, keys of a tile
constexpr int kSoftWarps = 8, kCopyWarp = 8, kMmaWarp = 9;
constexpr int kExpThreads = 320;
constexpr int kSmem = 227 * 1024 - 2048;
constexpr int kTmemCols = 512;
constexpr float kRaise = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Maps {
    CUtensorMap q_nope, q_rope, k_nope, k_rope, v;
};

// One thread's half row of a tile: the scores at tensor-memory address `col` (64
// columns, keys j0 ..; it sees those below lim) become weights, as bf16 in the
// first half of the same columns.  m: the row's reference, z: the thread's sum.
// The reference moves only when a row's maximum passes it by 2^8 (p stays below
// 2^8, which costs fp32 nothing): the two warps of these 32 rows then agree on a
// new one through `top` and rescale their rows of O, at `o` (DV / 2 columns a
// warp), after wait_o() -- the second product of the tile before.
template <int DV, typename WaitO>
__device__ __forceinline__ void softmax_half(uint32_t col, uint32_t o, int j0, int lim, float sl, bool first, int quarter,
                                             int half, int lane, float (*top)[32], float &m, float &z, const WaitO &wait_o)
{
    float x[64];
    ld32x32(&x[0], col);
    ld32x32(&x[32], col + 32);
    wait_ld();
    if (j0 + 64 > lim) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (j0 + i >= lim)
                x[i] = -CUDART_INF_F;
    }
    float part[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int i = 4; i < 64; ++i)
        part[i & 3] = fmaxf(part[i & 3], x[i]);
    const float mx = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])) * sl;
    // -inf + 8 is -inf: the first key that is seen raises it
    if (sync_any(1 + quarter, 64, first || mx > m + kRaise)) {
        top[half][lane] = mx;
        sync_some(1 + quarter, 64);
        const float all = fmaxf(mx, top[half ^ 1][lane]);
        float f = 1.0f;
        if (first) {
            m = all;
        } else if (all > m + kRaise) {
            f = ex2(m - all); // 0 from -inf: nothing is summed yet
            m = all;
            z *= f;
        }
        if (!first) {
            wait_o();
            fence_after();
#pragma unroll 1
            for (int c = 0; c < DV / 2; c += 32) {
                float v[32];
                ld32x32(v, o + uint32_t(DV / 2 * half + c));
                wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] *= f;
                st32x32(o + uint32_t(DV / 2 * half + c), v);
            }
            wait_st();
        }
        sync_some(1 + quarter, 64); // `top` is read
    }
    const float ref = m == -CUDART_INF_F ? 0.0f : m;
    float sum[4] = {};
    uint32_t p[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float e0 = ex2(fmaf(x[2 * i], sl, -ref)), e1 = ex2(fmaf(x[2 * i + 1], sl, -ref));
        sum[i & 3] += e0 + e1;
        p[i] = pack_bf16(e0, e1);
    }
    z += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    st32x32u(col, p); // over this thread's own scores
    wait_st();
}

// 32 columns of O at `o`, times inv (zeros where there is no O), as bf16 into a
// lane's row of `stage` (rows of `bytes` bytes), vectors v0 ..; swizzled, so that
// neither these stores nor reads by rows conflict.
__device__ __forceinline__ void stage32(uint8_t *stage, int bytes, uint32_t o, bool some, float inv, int v0, int lane)
{
    float v[32];
    if (some) {
        ld32x32(v, o);
        wait_ld();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (some) {
            u.x = pack_bf16(v[8 * i] * inv, v[8 * i + 1] * inv);
            u.y = pack_bf16(v[8 * i + 2] * inv, v[8 * i + 3] * inv);
            u.z = pack_bf16(v[8 * i + 4] * inv, v[8 * i + 5] * inv);
            u.w = pack_bf16(v[8 * i + 6] * inv, v[8 * i + 7] * inv);
        }
        *reinterpret_cast<uint4 *>(stage + lane * bytes + (((v0 + i) ^ (lane & 7)) << 4)) = u;
    }
}

// [toks][heads][cols] read in boxes of 64 columns x 1 head x `rows` tokens.
inline bool map_heads(CUtensorMap *m, const uint16_t *p, int toks, int heads, int cols, int64_t ld_tok, int64_t ld_head,
                      int rows)
{
    const uint64_t sizes[3] = {uint64_t(cols), uint64_t(heads), uint64_t(toks)};
    const uint64_t strides[2] = {uint64_t(ld_head) * 2, uint64_t(ld_tok) * 2};
    const uint32_t box[3] = {64, 1, uint32_t(rows)};
    return encode_bf16_map(m, p, 3, sizes, strides, box);
}
// All five, keys and values in boxes of k_rows and v_rows tokens.
inline bool map_all(Maps &maps, const w8_latent_expanded &a, int k_rows, int v_rows)
{
    bool ok = map_heads(&maps.q_nope, a.q_nope, a.n_q, a.n_heads, a.d_nope, a.ld_qnope_tok, a.ld_qnope_head, kRows) &&
              map_heads(&maps.q_rope, a.q_rope, a.n_q, a.n_heads, W8_LATENT_ROPE, a.ld_qrope_tok, a.ld_qrope_head, kRows);
    if (a.n_k > 0) { // without keys nothing is copied
        const uint64_t sizes[2] = {W8_LATENT_ROPE, uint64_t(a.n_k)}, strides[1] = {uint64_t(a.ld_krope_tok) * 2};
        const uint32_t box[2] = {64, uint32_t(k_rows)};
        ok = ok && map_heads(&maps.k_nope, a.k_nope, a.n_k, a.n_heads, a.d_nope, a.ld_knope_tok, a.ld_knope_head, k_rows) &&
             map_heads(&maps.v, a.v, a.n_k, a.n_heads, a.d_v, a.ld_v_tok, a.ld_v_head, v_rows) &&
             encode_bf16_map(&maps.k_rope, a.k_rope, 2, sizes, strides, box);
    } else {
        maps.k_nope = maps.v = maps.k_rope = maps.q_rope;
    }
    return ok;
}

} // namespace expanded

} // namespace w8
