// w8_latent_paged.cu -- latent attention, absorbed form, over the paged cache
// (w8_latent_attn_paged).
//
// The plainest form: a warp a (query token, head), one key after another, the
// running maximum and sum of the softmax beside the output in registers.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "w8_device.cuh"
#include "w8_serve_internal.h"

namespace w8 {

__device__ int g_serve_status;

namespace {

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }

__global__ void __launch_bounds__(256) paged_kernel(const w8_latent_paged a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= int64_t(a.n_tok) * a.n_heads)
        return;
    const int t = int(row / a.n_heads), h = int(row - int64_t(t) * a.n_heads);
    int r = 0;
    while (r < a.n_req && a.cu_q[r + 1] <= t)
        ++r;
    if (r == a.n_req || a.cu_q[r] > t)
        return;
    const int c0 = max(a.cu_q[r], 0), c1 = min(a.cu_q[r + 1], a.n_tok);
    const int64_t cap = int64_t(a.max_pages) * a.cache.page_size;
    const int len = int(min(int64_t(max(a.seq_lens[r], 0)), cap));
    const int last = len - (c1 - c0) + (t - c0); // the last key this token sees
    const uint16_t *ql = a.q_lat + t * a.ld_qlat_tok + h * a.ld_qlat_head;
    const uint16_t *qr = a.q_rope + t * a.ld_qrope_tok + h * a.ld_qrope_head;
    float q[18], acc[16] = {};
    for (int i = 0; i < 18; ++i)
        q[i] = i < 16 ? bf(ql[i * 32 + lane]) : bf(qr[(i - 16) * 32 + lane]);
    float m = -CUDART_INF_F, z = 0.0f;
    for (int j = 0; j <= last && j < len; ++j) {
        const int page = a.block_table[r * a.ld_table + j / a.cache.page_size];
        float k[18], x = 0.0f;
        for (int i = 0; i < 18; ++i) {
            k[i] = page >= 0 && page < a.cache.n_pages
                       ? bf(static_cast<const uint16_t *>(a.cache.data)[page * a.cache.ld_page + (j % a.cache.page_size) * a.cache.ld_tok +
                                                                        i * 32 + lane])
                       : 0.0f;
            x = fmaf(q[i], k[i], x);
        }
        for (int d = 16; d > 0; d >>= 1)
            x += __shfl_xor_sync(0xffffffffu, x, d);
        x *= a.scale;
        const float m1 = fmaxf(m, x), ref = m1 == -CUDART_INF_F ? 0.0f : m1; // NaN scores stay NaN
        const float f = expf(m - ref), p = expf(x - ref);
        m = m1;
        z = z * f + p;
        for (int i = 0; i < 16; ++i)
            acc[i] = fmaf(p, k[i], acc[i] * f);
    }
    for (int i = 0; i < 16; ++i) {
        const float o = z > 0.0f || z != z ? acc[i] / z : 0.0f;
        uint32_t u;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(0.0f), "f"(o));
        a.out[t * a.ld_out_tok + h * a.ld_out_head + i * 32 + lane] = uint16_t(u);
    }
    if (a.lse && lane == 0)
        a.lse[row] = (m == -CUDART_INF_F ? 0.0f : m) + logf(z);
}

} // namespace

size_t latent_paged_ws_bytes(int, int, int, int) { return 0; }

cudaError_t launch_latent_paged(const w8_latent_paged &a, void *, int, cudaStream_t s)
{
    const int64_t rows = int64_t(a.n_tok) * a.n_heads;
    return launch_dependent(&paged_kernel, dim3(unsigned((rows + 7) / 8)), 256, 0, s, a);
}

cudaError_t serve_status(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_serve_status, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_serve_status, &zero, sizeof(int));
    }
    return e;
}

} // namespace w8
