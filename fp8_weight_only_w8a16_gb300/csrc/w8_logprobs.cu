// w8_logprobs.cu -- log probability of a given token, entropy and the most
// likely alternatives, from one read of the logits (w8_token_logprobs).
//
// With m the row's maximum and d_v = x_v - m,
//   Z = sum exp(d_v),  W = sum exp(d_v) d_v:
//   lse = m + ln Z,  logprob(t) = d_t - ln Z,  entropy = ln Z - W / Z.
// (Z, W) relative to a smaller maximum m' become (Z, W) relative to m by
//   Z exp(m' - m)  and  exp(m' - m) (W + (m' - m) Z),
// so a thread keeps (m, Z, W) of what it has read and the threads', warps' and
// CTAs' results join in any grouping.  d is taken before the multiplication by
// log2 e (a difference of near values is exact, a product with a large logit
// is not).
//
// The alternatives: a logit's 32-bit value in order, then the inverted token
// number, make one 64-bit key, so all keys differ and equal logits rank by the
// lowest token.  A warp holds its best 32 keys sorted, one a lane; a vector of
// logits is looked at only when its maximum (needed for m anyway) passes the
// warp's `top`-th key, which for unordered logits happens about
// top ln(n / top) times over n logits.
//
// A row is cut into `splits` runs of whole 16-byte vectors, one a CTA; the
// last CTA of a row to arrive joins the runs in order of their number.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "w8_device.cuh"
#include "w8_serve_internal.h"

namespace w8 {

namespace {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpAhead = 4; // vectors a thread has in flight
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e38f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger of the two; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// m, Z and W; w in units of log2 until the row is finished.
struct Stat {
    float m, z, w;
};
// (0 x inf does not arise: e is 0 only with a delta that is cut at -1000)
__device__ __forceinline__ void stat_raise(Stat &s, float m)
{
    const float d = max_nan((s.m - m) * kLog2e, -1000.0f), e = ex2(d);
    s.w = e * (s.w + d * s.z);
    s.z *= e;
    s.m = m;
}
__device__ __forceinline__ void stat_join(Stat &s, Stat o)
{
    const float m = fmaxf(s.m, o.m);
    stat_raise(s, m);
    stat_raise(o, m);
    s.z += o.z;
    s.w += o.w;
}

// The order of floats as unsigned numbers (-0 with +0, NaN above +inf).
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    if (x != x)
        return 0xFFFFFFFFu;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o)
{
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, int token)
{
    return uint64_t(order_of(x)) << 32 | uint32_t(~token);
}
__device__ __forceinline__ int token_of(uint64_t key) { return int(~uint32_t(key)); }

// A warp's best keys, lane l the l-th; 0 where there is none yet.
struct Best {
    uint64_t key;  // this lane's
    uint64_t last; // the `top`-th
};
// Offers one key a lane (0: none).
__device__ __forceinline__ void best_offer(Best &b, uint64_t key, int top, int lane)
{
    uint32_t who;
    while ((who = __ballot_sync(0xffffffffu, key > b.last)) != 0) {
        const int src = __ffs(int(who)) - 1;
        const uint64_t k = __shfl_sync(0xffffffffu, key, src);
        const int at = __popc(__ballot_sync(0xffffffffu, b.key > k));
        const uint64_t up = __shfl_up_sync(0xffffffffu, b.key, 1);
        b.key = lane < at ? b.key : lane == at ? k : up;
        b.last = __shfl_sync(0xffffffffu, b.key, top - 1);
        if (lane == src)
            key = 0;
    }
}

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void widen(float (&x)[8], const uint4 &v)
    {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ float one(const void *p, int64_t i)
    {
        return __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t *>(p) + i)) << 16);
    }
};
template <>
struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void widen(float (&x)[4], const uint4 &v)
    {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float one(const void *p, int64_t i)
    {
        return __ldg(static_cast<const float *>(p) + i);
    }
};

__device__ __forceinline__ uint4 ld_once(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// n logits x[], tokens t0 .. (those with t0 + i outside [lo, hi) left out).
template <bool kTop, int N>
__device__ __forceinline__ void take(Stat &s, Best &b, const float (&x)[N], int t0, bool all, int lo, int hi,
                                     int top, int lane, bool live)
{
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i)
        mx = fmaxf(mx, x[i]);
    if (live) {
        if (mx > s.m)
            stat_raise(s, mx);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float d = max_nan((x[i] - s.m) * kLog2e, -1000.0f), e = ex2(d);
            s.z += e;
            s.w = fmaf(e, d, s.w);
        }
    }
    if constexpr (kTop) {
        // no warp-mate's vector passes the `top`-th value: the usual case (a
        // later token of the same value would rank behind; while the list is
        // not full its last key is 0, whose value is NaN, so everything passes)
        const bool pass = live && !(mx <= value_of(uint32_t(b.last >> 32)));
        if (__any_sync(0xffffffffu, pass)) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                best_offer(b, pass && (all || (t0 + i >= lo && t0 + i < hi)) ? key_of(x[i], t0 + i) : 0, top, lane);
        }
    }
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LogprobsArgs a)
{
    constexpr int N = Vec<T>::n;
    __shared__ Stat s_stat[kLpWarps];
    __shared__ uint64_t s_key[kLpWarps][32];
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x / a.splits;
    const int split = int(blockIdx.x - row * a.splits);
    pdl_launch_dependents();
    pdl_wait();

    // the row as 16-byte vectors: vector v holds tokens v N - skew ..; the
    // first and the last may stick out of the row and are read one by one
    const T *x = static_cast<const T *>(a.x) + row * a.ld;
    const int skew = int((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int nvec = (a.vocab + skew + N - 1) / N;
    const int v0 = int(int64_t(split) * nvec / a.splits), v1 = int(int64_t(split + 1) * nvec / a.splits);
    Stat s{kLowest, 0.0f, 0.0f};
    Best b{0, 0};
    for (int base = v0; base < v1; base += kLpThreads * kLpAhead) {
        uint4 raw[kLpAhead];
#pragma unroll
        for (int k = 0; k < kLpAhead; ++k) {
            const int v = base + k * kLpThreads + tid, t0 = v * N - skew;
            raw[k] = make_uint4(0, 0, 0, 0);
            if (v < v1 && t0 >= 0 && t0 + N <= a.vocab)
                raw[k] = ld_once(x + t0);
        }
#pragma unroll
        for (int k = 0; k < kLpAhead; ++k) {
            const int v = base + k * kLpThreads + tid, t0 = v * N - skew;
            if (base + k * kLpThreads + (tid & ~31) >= v1)
                break; // nothing for the whole warp
            const bool live = v < v1, all = t0 >= 0 && t0 + N <= a.vocab;
            float f[N];
            Vec<T>::widen(f, raw[k]);
            if (live && !all) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    f[i] = t0 + i >= 0 && t0 + i < a.vocab ? Vec<T>::one(x, t0 + i) : -CUDART_INF_F;
            }
            take<kTop, N>(s, b, f, t0, all, 0, a.vocab, a.top, lane, live);
        }
    }

    // the warp's, then the CTA's result
    auto warp_join = [&](Stat &st) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            Stat o;
            o.m = __shfl_xor_sync(0xffffffffu, st.m, d);
            o.z = __shfl_xor_sync(0xffffffffu, st.z, d);
            o.w = __shfl_xor_sync(0xffffffffu, st.w, d);
            stat_join(st, o);
        }
    };
    auto cta_join = [&]() {
        warp_join(s);
        if (lane == 0)
            s_stat[warp] = s;
        if constexpr (kTop)
            s_key[warp][lane] = b.key;
        __syncthreads();
        if (warp == 0) {
            s = lane < kLpWarps ? s_stat[lane] : Stat{kLowest, 0.0f, 0.0f};
            warp_join(s);
            if constexpr (kTop)
                for (int w = 1; w < kLpWarps; ++w)
                    best_offer(b, lane < a.top ? s_key[w][lane] : 0, a.top, lane);
        }
    };
    cta_join();
    if (a.splits > 1) {
        LogprobsPart *parts = a.parts + row * a.splits;
        if (warp == 0) {
            if (lane == 0) {
                parts[split].m = s.m;
                parts[split].z = s.z;
                parts[split].w = s.w;
            }
            if (kTop && lane < a.top)
                parts[split].key[lane] = b.key;
            __threadfence();
        }
        __syncthreads();
        if (tid == 0)
            s_last = atomicAdd(a.counters + row, 1) == a.splits - 1;
        __syncthreads();
        if (!s_last)
            return;
        __threadfence();
        s = Stat{kLowest, 0.0f, 0.0f};
        b = Best{0, 0};
        for (int i = tid; i < a.splits; i += kLpThreads)
            stat_join(s, Stat{__ldcg(&parts[i].m), __ldcg(&parts[i].z), __ldcg(&parts[i].w)});
        if constexpr (kTop)
            for (int i = warp; i < a.splits; i += kLpWarps)
                best_offer(b, lane < a.top ? __ldcg(&parts[i].key[lane]) : 0, a.top, lane);
        cta_join();
        if (tid == 0)
            a.counters[row] = 0;
    }
    if (warp == 0) {
        const float logz = logf(s.z);
        if (lane == 0) {
            const int t = __ldg(a.tokens + row);
            a.logprob[row] = t >= 0 && t < a.vocab ? Vec<T>::one(x, t) - s.m - logz : CUDART_NAN_F;
            if (a.entropy)
                a.entropy[row] = logz - s.w * kLn2 / s.z;
        }
        if (kTop && lane < a.top) {
            a.top_ids[row * a.top + lane] = token_of(b.key);
            a.top_logprobs[row * a.top + lane] = value_of(uint32_t(b.key >> 32)) - s.m - logz;
        }
    }
}

} // namespace

int logprobs_splits(int rows, int vocab, int sms)
{
    if (rows > kLogprobsCounters)
        return 1;
    // about eight CTAs an SM, none with less than 1024 logits
    const int64_t want = (int64_t(sms) * 8 + rows - 1) / rows;
    const int64_t most = (int64_t(vocab) + 1023) / 1024;
    const int64_t s = want < most ? want : most;
    return int(s < 1 ? 1 : s > sms ? sms : s);
}

cudaError_t launch_logprobs(const LogprobsArgs &a, bool bf16, cudaStream_t s)
{
    const dim3 grid{unsigned(int64_t(a.rows) * a.splits)};
    auto *fn = bf16 ? (a.top ? &logprobs_kernel<__nv_bfloat16, true> : &logprobs_kernel<__nv_bfloat16, false>)
                    : (a.top ? &logprobs_kernel<float, true> : &logprobs_kernel<float, false>);
    return launch_dependent(fn, grid, kLpThreads, 0, s, a);
}

} // namespace w8
