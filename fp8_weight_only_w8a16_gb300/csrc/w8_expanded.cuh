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

// s += 0 * (a, b): NaN where a value is not finite.
__device__ __forceinline__ void add_times0(float2 &s, float a, float b)
{
    asm("{\n\t.reg .b64 v, t, z;\n\tmov.b64 v, {%2, %3};\n\tmov.b64 t, {%0, %1};\n\tmov.b64 z, 0;\n\t"
        "fma.rn.f32x2 t, v, z, t;\n\tmov.b64 {%0, %1}, t;\n\t}"
        : "+f"(s.x), "+f"(s.y)
        : "f"(a), "f"(b));
}

// 32 columns of O at `o`, times inv (zeros where there is no O), as bf16 into a
// lane's row of `stage` (rows of `bytes` bytes), vectors v0 ..; swizzled, so that
// neither these stores nor reads by rows conflict.  zero: 0, and NaN once a value is
// not finite.
__device__ __forceinline__ void stage32(uint8_t *stage, int bytes, uint32_t o, bool some, float inv, int v0, int lane, float &zero)
{
    float v[32];
    if (some) {
        ld32x32(v, o);
        wait_ld();
        float2 part[2] = {{zero, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
        for (int i = 0; i < 16; ++i)
            add_times0(part[i & 1], v[2 * i], v[2 * i + 1]);
        zero = (part[0].x + part[0].y) + (part[1].x + part[1].y);
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

__device__ __forceinline__ float2 widen2(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)); }
// Rows of an operand in words of two values, from a token and head on.
struct Words {
    const uint32_t *p;
    int64_t ld;
    __device__ __forceinline__ Words(const uint16_t *from, int64_t tok, int64_t ld_tok, int64_t column)
        : p(reinterpret_cast<const uint32_t *>(from + tok * ld_tok + column)), ld(ld_tok / 2)
    {
    }
    __device__ __forceinline__ uint32_t at(int tok, int i) const { return __ldg(p + tok * ld + i); }
};

// Causality hides keys from some rows of a tile: their weights there are 0, but
// 0 x NaN is not, nor 0 x infinity.  So rows whose output is not finite although
// their sum of weights is, and which do not see all keys, are looked at again by a
// warp: where a value among the keys below `end` that is hidden from a row is not
// finite, the row's output is made once more from the keys it sees, one at a time.
// (No input of finite values comes here: searching the values before every diagonal
// tile's second product would hold that up.  A prompt of 4096 at 64 heads: 386 us, one
// value that all see NaN 600, half of all 956, all of them 1350.  A key of a row takes
// 0.1 us; the other warps wait up to 5 s, or 1.6 million keys for 32 rows.)  bad: such
// rows of this warp's 32, lane i's being query q0 + i with `lim` keys, reference m, sum z; the
// warp's columns are d_v / 2 of them from DV / 2 * half on.
template <int DN, int DV>
__device__ __noinline__ void redo_rows(const w8_latent_expanded &a, uint32_t bad, int q0, int head, int k0, int end, int lim, float m,
                                       float z, int half, int lane)
{
    constexpr int kQ = DN / 64, kV = DV / 128; // words of 2 values a lane
    const float sl = a.scale * kLog2e;
    const Words qn(a.q_nope, q0, a.ld_qnope_tok, head * a.ld_qnope_head + 2 * lane),
        qr(a.q_rope, q0, a.ld_qrope_tok, head * a.ld_qrope_head + 2 * lane),
        kn(a.k_nope, k0, a.ld_knope_tok, head * a.ld_knope_head + 2 * lane), kr(a.k_rope, k0, a.ld_krope_tok, 2 * lane),
        v(a.v, k0, a.ld_v_tok, head * a.ld_v_head + DV / 2 * half + 2 * lane);
    uint16_t *const out = a.out + int64_t(q0) * a.ld_out_tok + head * a.ld_out_head + DV / 2 * half + 2 * lane;
    const int64_t ld_out = a.ld_out_tok;
    // the last hidden key whose value is not finite in the warp's columns
    int last = -1;
    for (int j = __reduce_min_sync(0xffffffffu, bad >> lane & 1u ? lim : INT32_MAX); j < end; ++j) {
        bool inf = false;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const uint32_t u = v.at(j, 32 * i);
            inf = inf || (u & 0x7F80u) == 0x7F80u || (u & 0x7F800000u) == 0x7F800000u;
        }
        if (__any_sync(0xffffffffu, inf))
            last = j;
    }
    bad &= __ballot_sync(0xffffffffu, lim <= last);
    for (; bad; bad &= bad - 1) {
        const int row = __ffs(int(bad)) - 1, keys = __shfl_sync(0xffffffffu, lim, row);
        const float at = __shfl_sync(0xffffffffu, m, row), sum = __shfl_sync(0xffffffffu, z, row);
        const float ref = at == -CUDART_INF_F ? 0.0f : at;
        float2 q[kQ + 1], o[kV] = {};
#pragma unroll
        for (int i = 0; i < kQ; ++i)
            q[i] = widen2(qn.at(row, 32 * i));
        q[kQ] = widen2(qr.at(row, 0));
        // from the last key back, some at a time, until all is NaN: a row that sees such
        // values mostly does so near its end
        constexpr int kAtOnce = 8;
        bool left = true;
        for (int j1 = keys; j1 > 0 && left; j1 -= kAtOnce) {
            float p[kAtOnce];
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int j = max(j1 - 1 - n, 0);
                float2 b = widen2(kr.at(j, 0));
                p[n] = fmaf(q[kQ].x, b.x, q[kQ].y * b.y);
#pragma unroll
                for (int i = 0; i < kQ; ++i) {
                    b = widen2(kn.at(j, 32 * i));
                    p[n] = fmaf(q[i].x, b.x, fmaf(q[i].y, b.y, p[n]));
                }
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
#pragma unroll
                for (int n = 0; n < kAtOnce; ++n)
                    p[n] += __shfl_xor_sync(0xffffffffu, p[n], d);
            bool nan = true;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
#pragma unroll
                for (int n = 0; n < kAtOnce; ++n)
                    if (n < j1) {
                        const float2 b = widen2(v.at(j1 - 1 - n, 32 * i));
                        const float w = ex2(fmaf(p[n], sl, -ref));
                        o[i].x = fmaf(w, b.x, o[i].x);
                        o[i].y = fmaf(w, b.y, o[i].y);
                    }
                nan = nan && o[i].x != o[i].x && o[i].y != o[i].y;
            }
            left = !__all_sync(0xffffffffu, nan);
        }
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i)
            *reinterpret_cast<uint32_t *>(out + row * ld_out + 64 * i) = pack_bf16(o[i].x * inv, o[i].y * inv);
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
