// w8_latent_expanded.cu -- latent attention, expanded form, over the keys and
// values of a prompt (w8_latent_attn_expanded).
//
// The plainest form: a warp a (query token, head), one key after another, the
// running maximum and sum of the softmax beside the output in registers.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "w8_device.cuh"
#include "w8_serve_internal.h"

namespace w8 {

namespace {

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }

template <int DN, int DV>
__global__ void __launch_bounds__(256) expanded_kernel(const w8_latent_expanded a)
{
    constexpr int NQ = (DN + 64) / 32, NV = DV / 32;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= int64_t(a.n_q) * a.n_heads)
        return;
    const int t = int(row / a.n_heads), h = int(row - int64_t(t) * a.n_heads);
    int r = 0;
    while (r < a.n_req && a.cu_q[r + 1] <= t)
        ++r;
    if (r == a.n_req || a.cu_q[r] > t)
        return;
    const int q0 = max(a.cu_q[r], 0), q1 = min(a.cu_q[r + 1], a.n_q);
    const int k0 = min(max(a.cu_k[r], 0), a.n_k), k1 = min(max(a.cu_k[r + 1], k0), a.n_k);
    const int last = a.causal ? (k1 - k0) - (q1 - q0) + (t - q0) : k1 - k0 - 1;
    float q[NQ], acc[NV] = {};
    for (int i = 0; i < NQ; ++i)
        q[i] = i < DN / 32 ? bf(a.q_nope[t * a.ld_qnope_tok + h * a.ld_qnope_head + i * 32 + lane])
                           : bf(a.q_rope[t * a.ld_qrope_tok + h * a.ld_qrope_head + (i - DN / 32) * 32 + lane]);
    float m = -CUDART_INF_F, z = 0.0f;
    for (int j = k0; j <= k0 + last && j < k1; ++j) {
        float x = 0.0f;
        for (int i = 0; i < NQ; ++i) {
            const float k = i < DN / 32 ? bf(a.k_nope[j * a.ld_knope_tok + h * a.ld_knope_head + i * 32 + lane])
                                        : bf(a.k_rope[j * a.ld_krope_tok + (i - DN / 32) * 32 + lane]);
            x = fmaf(q[i], k, x);
        }
        for (int d = 16; d > 0; d >>= 1)
            x += __shfl_xor_sync(0xffffffffu, x, d);
        x *= a.scale;
        const float m1 = fmaxf(m, x), ref = m1 == -CUDART_INF_F ? 0.0f : m1; // NaN scores stay NaN
        const float f = expf(m - ref), p = expf(x - ref);
        m = m1;
        z = z * f + p;
        for (int i = 0; i < NV; ++i)
            acc[i] = fmaf(p, bf(a.v[j * a.ld_v_tok + h * a.ld_v_head + i * 32 + lane]), acc[i] * f);
    }
    for (int i = 0; i < NV; ++i) {
        const float o = z > 0.0f || z != z ? acc[i] / z : 0.0f;
        uint32_t u;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(0.0f), "f"(o));
        a.out[t * a.ld_out_tok + h * a.ld_out_head + i * 32 + lane] = uint16_t(u);
    }
    if (a.lse && lane == 0)
        a.lse[row] = (m == -CUDART_INF_F ? 0.0f : m) + logf(z);
}

} // namespace

cudaError_t expanded_status(int *out, bool)
{
    *out = 0;
    return cudaSuccess;
}

cudaError_t launch_latent_expanded(const w8_latent_expanded &a, int, cudaStream_t s)
{
    const int64_t rows = int64_t(a.n_q) * a.n_heads;
    auto *fn = a.d_nope == 192 ? &expanded_kernel<192, 256> : &expanded_kernel<128, 128>;
    return launch_dependent(fn, dim3(unsigned((rows + 7) / 8)), 256, 0, s, a);
}

} // namespace w8
