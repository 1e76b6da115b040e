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
// lowest token.  A thread keeps the largest value of what it has read (the sums
// need the vectors' maxima anyway).  From the threads' largest values comes a
// bound that at least `top` logits reach; the few threads that reach it have
// their vectors read once more, the keys that pass are gathered, and a key's
// place is the number of larger keys gathered.  The loop over the logits knows
// nothing of the selection.
//
// Measured (replayed, 154880 logits): 1024 bf16 rows with 1 alternative 59 to 61
// us, 5.3 TB/s (without alternatives 53, fp32 94 us = 6.7 TB/s: HBM); 48 fp32 rows
// with 20 alternatives 15 us, one bf16 row with 5 alternatives 8.7 us, without
// 4.3: the selection and the join are chains of a few us that only many rows
// hide.  bf16 is at 62 % of the issue slots, six instructions a logit.
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
constexpr int kLpAhead = 4; // vectors a thread has in flight beside those it works on
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e38f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// Two floats in one register pair.
__device__ __forceinline__ uint64_t pair_of(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 pair_values(uint64_t p)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 16 bytes of logits: their number, values, largest and smallest (of those
// that are not NaN).
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
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    template <int K>
    static __device__ __forceinline__ void range(float &lo, float &hi, const uint4 (&v)[K])
    {
        uint32_t a = v[0].x, b = v[0].x;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            a = max2(a, max2(max2(v[k].x, v[k].y), max2(v[k].z, v[k].w)));
            b = min2(b, min2(min2(v[k].x, v[k].y), min2(v[k].z, v[k].w)));
        }
        hi = fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
        lo = fminf(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u));
    }
    static __device__ __forceinline__ float one(const void *p, int64_t i)
    {
        return __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t *>(p) + i)) << 16);
    }
    static __device__ __forceinline__ float held(const void *p, int i)
    {
        return __uint_as_float(uint32_t(static_cast<const uint16_t *>(p)[i]) << 16);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8])
    {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = __float_as_uint(x[2 * i]) >> 16 | (__float_as_uint(x[2 * i + 1]) & 0xFFFF0000u);
        return make_uint4(u[0], u[1], u[2], u[3]);
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
    template <int K>
    static __device__ __forceinline__ void range(float &lo, float &hi, const uint4 (&v)[K])
    {
        lo = hi = __uint_as_float(v[0].x);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float x[4];
            widen(x, v[k]);
            hi = fmaxf(hi, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
            lo = fminf(lo, fminf(fminf(x[0], x[1]), fminf(x[2], x[3])));
        }
    }
    static __device__ __forceinline__ float one(const void *p, int64_t i)
    {
        return __ldg(static_cast<const float *>(p) + i);
    }
    static __device__ __forceinline__ float held(const void *p, int i) { return static_cast<const float *>(p)[i]; }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
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

// The sums take in K vectors; `z` and `w` in pairs.  hi: their largest value.
template <typename T, int K>
__device__ __forceinline__ void take(Stat &s, uint64_t &z, uint64_t &w, const uint4 (&raw)[K], float &hi)
{
    constexpr int N = Vec<T>::n;
    float lo;
    Vec<T>::range(lo, hi, raw);
    if (hi > s.m) { // a new reference
        const float2 a = pair_values(z), b = pair_values(w);
        s.z = a.x + a.y;
        s.w = b.x + b.y;
        stat_raise(s, hi);
        z = pair_of(s.z, 0.0f);
        w = pair_of(s.w, 0.0f);
    }
    const uint64_t minus = pair_of(-s.m, -s.m), scale = pair_of(kLog2e, kLog2e);
    if ((lo - s.m) * kLog2e >= -1000.0f) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float x[N];
            Vec<T>::widen(x, raw[k]);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const uint64_t d = pair_mul(pair_add(pair_of(x[i], x[i + 1]), minus), scale);
                const float2 v = pair_values(d);
                const uint64_t e = pair_of(ex2(v.x), ex2(v.y));
                z = pair_add(z, e);
                w = pair_fma(e, d, w);
            }
        }
    } else { // banned tokens, or a masked value far below: 0 x infinity is kept out of w
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float x[N];
            Vec<T>::widen(x, raw[k]);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float d0 = max_nan((x[i] - s.m) * kLog2e, -1000.0f), d1 = max_nan((x[i + 1] - s.m) * kLog2e, -1000.0f);
                const uint64_t e = pair_of(ex2(d0), ex2(d1));
                z = pair_add(z, e);
                w = pair_fma(e, pair_of(d0, d1), w);
            }
        }
    }
}

// Gathered keys, and what the selection shares.
constexpr int kGather = 256;
struct Select {
    uint64_t key[kGather];
    uint64_t best[W8_MAX_TOP];
    uint64_t bound;      // keys from here on are gathered,
    uint64_t loose;      // or from here on, if those are too few (0: they are not)
    uint32_t nth[kLpWarps];
    int count, passing;
    uint8_t thread[kLpThreads]; // those whose largest value reaches the bound
};

// best[0 .. top - 1] = the largest of the keys that `scan` offers, in falling
// order (0 where there are fewer), over all threads of the CTA.  scan(offer)
// calls offer(key) for every key that may count, and offers the same keys
// whenever it is called; at least `top` of them, if there are that many, reach
// sel.bound, or else sel.loose.  When more pass than there is room for, the `top`-th of those
// gathered is the next bound: an eighth of them or less pass it.
template <typename Scan>
__device__ __forceinline__ void select_top(Select &sel, int top, int tid, const Scan &scan)
{
    for (;;) {
        if (tid == 0)
            sel.count = 0;
        if (tid < top)
            sel.best[tid] = 0;
        __syncthreads();
        const uint64_t bound = sel.bound;
        scan([&](uint64_t key) {
            if (key >= bound && key != 0) {
                const int at = atomicAdd(&sel.count, 1);
                if (at < kGather)
                    sel.key[at] = key;
            }
        });
        __syncthreads();
        const int n = min(sel.count, kGather);
        const bool more = sel.count > kGather, few = n < top && sel.loose != 0;
        if (tid < n) {
            const uint64_t mine = sel.key[tid];
            int rank = 0;
            for (int i = 0; i < n; ++i)
                rank += sel.key[i] > mine;
            if (rank < top)
                sel.best[rank] = mine;
        }
        __syncthreads();
        if (!more && !few)
            return;
        if (tid == 0) {
            sel.bound = few ? sel.loose : sel.best[top - 1];
            sel.loose = 0;
        }
        __syncthreads();
    }
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_kernel(const LogprobsArgs a)
{
    constexpr int N = Vec<T>::n;
    __shared__ Stat s_stat[kLpWarps];
    __shared__ Select sel;
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
    const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u; // -inf
    // any vector, -inf where the row has no token
    auto load = [&](int v) {
        const int t0 = v * N - skew;
        if (t0 >= 0 && t0 + N <= a.vocab)
            return ld_once(x + t0);
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] = t0 + i >= 0 && t0 + i < a.vocab ? Vec<T>::one(x, t0 + i) : -CUDART_INF_F;
        return Vec<T>::pack(f);
    };
    Stat s{kLowest, 0.0f, 0.0f};
    uint64_t z = pair_of(0.0f, 0.0f), w = z;
    float top_value = CUDART_NAN_F; // the largest read so far; passed by anything at first
    {
        // the run's vectors that lie inside the row: f0 .. f1 - 1, thread tid
        // those at v0 + tid, + 256, ..; the next ones are on their way while
        // these are taken in
        const int f0 = max(v0, skew ? 1 : 0), f1 = min(v1, (a.vocab + skew) / N);
        const uint32_t inside = uint32_t(max(f1 - f0, 0));
        const uint8_t *p = reinterpret_cast<const uint8_t *>(x - skew) + int64_t(v0 + tid) * 16;
        uint4 raw[kLpAhead];
        auto fetch = [&](int at) { // at: the first one's place from f0
#pragma unroll
            for (int k = 0; k < kLpAhead; ++k) {
                raw[k] = make_uint4(none, none, none, none);
                if (uint32_t(at + k * kLpThreads) < inside)
                    raw[k] = ld_once(p + k * kLpThreads * 16);
            }
            p += kLpAhead * kLpThreads * 16;
        };
        int at = v0 + tid - f0;
        fetch(at);
        for (; at < int(inside); at += kLpAhead * kLpThreads) {
            uint4 now[kLpAhead];
#pragma unroll
            for (int k = 0; k < kLpAhead; ++k)
                now[k] = raw[k];
            fetch(at + kLpAhead * kLpThreads);
            float hi;
            take<T>(s, z, w, now, hi);
            if (kTop && !(hi <= top_value))
                top_value = hi;
        }
        // the vectors that stick out of the row
        for (int e = 0; e < 2; ++e) {
            const int v = e ? nvec - 1 : 0;
            if (v >= v0 && v < v1 && (v < f0 || v >= f1) && (e == 0 || nvec > 1) && (v - v0) % kLpThreads == tid) {
                const uint4 edge[1] = {load(v)};
                float hi;
                take<T>(s, z, w, edge, hi);
                if (kTop && !(hi <= top_value))
                    top_value = hi;
            }
        }
    }
    {
        const float2 zz = pair_values(z), ww = pair_values(w);
        s.z = zz.x + zz.y;
        s.w = ww.x + ww.y;
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
    auto cta_join = [&]() { // into warp 0
        warp_join(s);
        if (lane == 0)
            s_stat[warp] = s;
        __syncthreads();
        if (warp == 0) {
            s = lane < kLpWarps ? s_stat[lane] : Stat{kLowest, 0.0f, 0.0f};
            warp_join(s);
        }
    };
    cta_join();
    if constexpr (kTop) {
        // The bound: of the warps' k-th largest values (k = top / warps, rounded
        // up), the c-th largest, c k >= top.  Warps that are not full of vectors
        // have no say; without a full one (under 32 vectors) everything passes.
        const int nv = v1 - v0, full = min(nv / 32, kLpWarps);
        const uint32_t mine = tid < nv ? order_of(top_value) : 0;
        uint64_t bound = 0;
        if (full > 0) {
            const int k = (a.top + full - 1) / full, c = (a.top + k - 1) / k;
            uint32_t left = mine, nth = 0;
            for (int i = 0; i < k; ++i) {
                nth = __reduce_max_sync(0xffffffffu, left);
                const uint32_t who = __ballot_sync(0xffffffffu, left == nth);
                if (lane == __ffs(int(who)) - 1)
                    left = 0;
            }
            if (lane == 0)
                sel.nth[warp] = nth;
            __syncthreads();
            uint32_t own = lane < full ? sel.nth[lane] : 0;
            int rank = 0;
            for (int i = 0; i < full; ++i) {
                const uint32_t o = __shfl_sync(0xffffffffu, own, i);
                rank += o > own || (o == own && i < lane);
            }
            const uint32_t at = __ballot_sync(0xffffffffu, lane < full && rank == c - 1);
            bound = uint64_t(__shfl_sync(0xffffffffu, own, __ffs(int(at)) - 1)) << 32;
        }
        if (tid == 0) {
            sel.bound = bound;
            sel.loose = 0;
            sel.passing = 0;
        }
        __syncthreads();
        if (tid < nv && uint64_t(mine) << 32 >= bound)
            sel.thread[atomicAdd(&sel.passing, 1)] = uint8_t(tid);
        __syncthreads();
        // Where every thread reaches the bound it is most likely the value of
        // nearly all tokens, a mask's: the larger ones and, of its own, the run's
        // first 224 will do.  (48 rows of 154880 bf16 of which 155 are not
        // masked, 32 alternatives: 28 us; with all that reach it gathered, 113.)
        if (tid == 0 && bound != 0 && sel.passing == min(nv, kLpThreads)) {
            sel.loose = bound;
            sel.bound = bound | uint32_t(~(max(v0 * N - skew, 0) + 223));
        }
        __syncthreads();
        const int per = (nv + kLpThreads - 1) / kLpThreads, pairs = sel.passing * per;
        select_top(sel, a.top, tid, [&](auto &&offer) {
            const float least = value_of(uint32_t(sel.bound >> 32));
            for (int i0 = tid; i0 < pairs; i0 += kLpAhead * kLpThreads) {
                uint4 u[kLpAhead][1]; // all on their way before the first is looked at
                int t0[kLpAhead];
#pragma unroll
                for (int q = 0; q < kLpAhead; ++q) {
                    const int i = i0 + q * kLpThreads, j = i / per;
                    u[q][0] = make_uint4(none, none, none, none);
                    t0[q] = a.vocab;
                    if (i < pairs) {
                        const int v = v0 + (i - j * per) * kLpThreads + sel.thread[j];
                        if (v < v1) {
                            u[q][0] = load(v);
                            t0[q] = v * N - skew;
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < kLpAhead; ++q) {
                    float lo, hi, f[N];
                    Vec<T>::range(lo, hi, u[q]);
                    if (hi < least)
                        continue;
                    Vec<T>::widen(f, u[q][0]);
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (t0[q] + e >= 0 && t0[q] + e < a.vocab)
                            offer(key_of(f[e], t0[q] + e));
                }
            }
        });
    }
    if (a.splits > 1) {
        LogprobsPart *parts = a.parts + row * a.splits;
        if (warp == 0) {
            if (lane == 0) {
                parts[split].m = s.m;
                parts[split].z = s.z;
                parts[split].w = s.w;
            }
            if (kTop && lane < a.top)
                parts[split].key[lane] = sel.best[lane];
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
        for (int i = tid; i < a.splits; i += kLpThreads)
            stat_join(s, Stat{__ldcg(&parts[i].m), __ldcg(&parts[i].z), __ldcg(&parts[i].w)});
        if constexpr (kTop) {
            // the bound: of the runs' d-th keys, d = top / runs rounded up, the c-th largest, c d >= top
            const int d = (a.top + a.splits - 1) / a.splits, c = (a.top + d - 1) / d;
            for (int i = tid; i < a.splits; i += kLpThreads)
                sel.key[i] = __ldcg(&parts[i].key[d - 1]);
            __syncthreads();
            if (tid < a.splits) {
                const uint64_t mine = sel.key[tid];
                int rank = 0;
                for (int i = 0; i < a.splits; ++i)
                    rank += sel.key[i] > mine || (sel.key[i] == mine && i < tid); // equal ones are empty
                if (rank == c - 1) {
                    sel.bound = mine;
                    sel.loose = 0;
                }
            }
            __syncthreads();
            select_top(sel, a.top, tid, [&](auto &&offer) {
#pragma unroll 4
                for (int i = tid; i < a.splits * a.top; i += kLpThreads)
                    offer(__ldcg(&parts[i / a.top].key[i % a.top]));
            });
        }
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
            // a place that is left (a row of NaN) gets a token all the same
            const uint64_t key = sel.best[lane];
            a.top_ids[row * a.top + lane] = key ? token_of(key) : lane;
            a.top_logprobs[row * a.top + lane] = key ? value_of(uint32_t(key >> 32)) - s.m - logz : CUDART_NAN_F;
        }
    }
}

} // namespace

int logprobs_splits(int rows, int vocab, int sms)
{
    if (rows > kLogprobsCounters)
        return 1;
    // One wave of CTAs, four an SM, none with less than 4096 logits: a CTA's
    // selection and the join cost a few us that a second wave pays again.  Of
    // 154880 bf16 logits, 5 alternatives: 48 rows in 12 runs 12.4 us, in 25
    // runs 19.2; 1 row in 38 runs 8.7 us, in 152 runs 11.2; 1024 rows in 1 run
    // each 60.8 us, in 4 runs 81.5 (1 alternative).
    const int64_t want = int64_t(sms) * 4 / rows, most = (int64_t(vocab) + 4095) / 4096;
    const int64_t s = want < most ? want : most;
    return int(s < 1 ? 1 : s > kGather ? kGather : s);
}

cudaError_t launch_logprobs(const LogprobsArgs &a, bool bf16, cudaStream_t s)
{
    const dim3 grid{unsigned(int64_t(a.rows) * a.splits)};
    auto *fn = bf16 ? (a.top ? &logprobs_kernel<__nv_bfloat16, true> : &logprobs_kernel<__nv_bfloat16, false>)
                    : (a.top ? &logprobs_kernel<float, true> : &logprobs_kernel<float, false>);
    return launch_dependent(fn, grid, kLpThreads, 0, s, a);
}

} // namespace w8
