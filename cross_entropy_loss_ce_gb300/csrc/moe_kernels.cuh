// A router's balance loss and z-loss with per-expert counts and the gradient
// of its logits x [T, E], the experts each token was sent to given.
//
// With f_e the number of slots that chose expert e, n the counted tokens, k
// slots a token, p_t = softmax(x_t) and lse_t its log-sum-exp:
//   L       = a E / (k n^2) sum_t sum_e f_e p_te + b / n sum_t lse_t^2
//   dL/dx_te = p_te (a E / (k n^2) (f_e - sum_j p_tj f_j) + 2 b / n lse_t)
// (the first term is a E sum_e (f_e / (k n)) mean_t p_te, 1 a when tokens are
// spread evenly).  sum_j p_tj = 1, so any constant may be taken from f: the
// kernels use f_e less its mean, which keeps the small difference of two large
// counts out of the rounding.
//
// The counts need every token before the first gradient can be formed, but not
// the logits: moe_count_kernel reads the choices (integer atomics, so the
// order is free) and moe_rows_kernel then reads each row of logits once, into
// registers, and writes its gradient once.  A row belongs to 4 to 32 lanes;
// each lane keeps the counts of its experts in registers over all its rows and
// has the next row's loads in flight while it works on one.  Row losses are
// added in fp32 with their rounding errors carried (Neumaier) in an order fixed
// by the grid; the last CTA to finish adds the CTAs' sums in fp64.
#pragma once

#include "row_kernels.cuh"

namespace gbce {

constexpr int kMoeThreads = 256;
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxSlots = 64;
constexpr int kMoeMaxCtas = 2048;
constexpr float kMoeFar = 1048576.f;  // logits from here on are taken about their row's maximum first

// Zeroed before a moe_count_kernel of several CTAs.
struct MoeTotals {
    unsigned long long counts[kMoeMaxExperts];
    unsigned int n, bad, done, pad;
};

struct MoeArgs {
    const void *logits;
    int64_t ls;
    const int64_t *experts;
    int64_t es;
    int64_t T;
    int E, k;
    MoeTotals *totals;
    unsigned char *mask;   // [T]: the token counts (one CTA: in its shared memory)
    double *part;          // [gridDim.x] sums of row losses
    int64_t *counts;       // out
    float *loss;           // out, or NULL
    void *grad;            // out, or NULL
    int64_t gs;
    const float *grad_scale;
    float balance, z;
};

// Adds the choices of tokens first, first + step, ... to hist; returns how many
// count, i.e. have a slot in [0, E) and none beyond.  Up to 8 slots are loaded at
// once and kept; further ones are read again to be counted.
__device__ __forceinline__ int moe_count_tokens(const MoeArgs &a, int64_t first, int64_t step,
                                                unsigned *hist, unsigned char *mask, bool &bad)
{
    int n = 0;
    for (int64_t t = first; t < a.T; t += step) {
        const int64_t *ids = a.experts + t * a.es;
        int64_t e[8];
        bool any = false, wrong = false;
        const auto look = [&](int j0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                e[j] = j0 + j < a.k ? __ldg(ids + j0 + j) : -1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                any |= e[j] >= 0;
                wrong |= e[j] < -1 || e[j] >= a.E;
            }
        };
        for (int j0 = 8; j0 < a.k; j0 += 8)
            look(j0);
        look(0);
        const bool counted = any && !wrong;
        mask[t] = counted;
        bad |= wrong;
        n += counted;
        for (int j0 = 0; counted && j0 < a.k; j0 += 8) {
            if (j0)
                look(j0);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e[j] >= 0)
                    atomicAdd(hist + e[j], 1u);
        }
    }
    return n;
}

template <int NT>
__global__ void __launch_bounds__(NT) moe_count_kernel(const MoeArgs a)
{
    __shared__ unsigned hist[kMoeMaxExperts];
    __shared__ int all, wrong;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0)
        all = wrong = 0;
    for (int e = threadIdx.x; e < a.E; e += NT)
        hist[e] = 0;
    __syncthreads();
    bool bad = false;
    int n = moe_count_tokens(a, blockIdx.x * int64_t{NT} + threadIdx.x, int64_t{gridDim.x} * NT, hist, a.mask, bad);
    n = __reduce_add_sync(0xffffffffu, n);
    if (bad)
        atomicOr(&g_flags, kFlagBadTarget);
    if (gridDim.x == 1) {  // nothing to add to: no zeroing before
        if ((threadIdx.x & 31) == 0 && n)
            atomicAdd(&all, n);
        if (bad)
            wrong = 1;
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += NT)
            a.totals->counts[e] = hist[e];
        if (threadIdx.x == 0) {
            a.totals->n = static_cast<unsigned>(all);
            a.totals->bad = static_cast<unsigned>(wrong);
            a.totals->done = 0u;
        }
        return;
    }
    if ((threadIdx.x & 31) == 0 && n)
        atomicAdd(&a.totals->n, static_cast<unsigned>(n));
    if (bad)
        atomicOr(&a.totals->bad, 1u);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += NT)
        if (hist[e])
            atomicAdd(&a.totals->counts[e], static_cast<unsigned long long>(hist[e]));
}

template <int LPT>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

template <int LPT>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// VEC values of a row as they lie in memory: 16 or 8 bytes, or one value.
template <typename T, int VEC>
struct MoeUnit {
    using Raw = std::conditional_t<VEC == 1, T, std::conditional_t<VEC * sizeof(T) == 16, uint4, uint2>>;
    __device__ static __forceinline__ Raw load(const T *p)
    {
        if constexpr (VEC == 1)
            return *p;
        else
            return __ldcs(reinterpret_cast<const Raw *>(p));
    }
    __device__ static __forceinline__ void unpack(const Raw &r, float *f)
    {
        if constexpr (VEC == 1) {
            f[0] = Elem<T>::load(&r);
        } else {
            float v[Elem<T>::kPerVec];
            if constexpr (sizeof(Raw) == 16)
                Elem<T>::unpack(r, v);
            else
                Elem<T>::unpack(make_uint4(r.x, r.y, 0, 0), v);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                f[i] = v[i];
        }
    }
    __device__ static __forceinline__ void store(T *p, const float *f)
    {
        if constexpr (VEC == 1) {
            Elem<T>::store(p, f[0]);
        } else {
            float v[Elem<T>::kPerVec] = {};
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                v[i] = f[i];
            const uint4 r = Elem<T>::pack(v);
            if constexpr (sizeof(Raw) == 16)
                __stcs(reinterpret_cast<uint4 *>(p), r);
            else
                __stcs(reinterpret_cast<uint2 *>(p), make_uint2(r.x, r.y));
        }
    }
};

constexpr int kMoeSmallTokens = 256;  // tokens up to which one CTA does everything

// ALL: one CTA does everything, the counting too (small batches: one launch).
template <typename T, int VEC, int LPT, int NJ, bool ALL, int NT>
__global__ void __launch_bounds__(NT) moe_rows_kernel(const MoeArgs a)
{
    using Unit = MoeUnit<T, VEC>;
    __shared__ unsigned hist[ALL ? kMoeMaxExperts : 1];
    __shared__ unsigned char small_mask[ALL ? kMoeSmallTokens : 1];
    __shared__ float centred[kMoeMaxExperts];
    __shared__ long long warp_sum64[NT / 32];
    __shared__ double warp_part[NT / 32];
    __shared__ int s_n, s_bad, s_last;
    const int lane = threadIdx.x & 31, sub = lane % LPT;
    const int64_t groups = int64_t{gridDim.x} * (NT / LPT);
    int64_t t = blockIdx.x * int64_t{NT / LPT} + threadIdx.x / LPT;
    const T *logits = static_cast<const T *>(a.logits);
    const unsigned char *mask = ALL ? small_mask : a.mask;

    // the row's values as loaded; the first ones before the counts are needed
    typename Unit::Raw raw[NJ];
    const auto load_row = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = (j * LPT + sub) * VEC;
            if (row < a.T && e < a.E)
                raw[j] = Unit::load(logits + row * a.ls + e);
        }
    };
    load_row(t);

    if constexpr (ALL) {
        for (int e = threadIdx.x; e < a.E; e += NT)
            hist[e] = 0;
        if (threadIdx.x == 0)
            s_n = s_bad = 0;
        __syncthreads();
        bool bad = false;
        int n = moe_count_tokens(a, threadIdx.x, NT, hist, small_mask, bad);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0 && n)
            atomicAdd(&s_n, n);
        if (bad)
            s_bad = 1;
        __syncthreads();
        if (threadIdx.x == 0 && s_bad)
            atomicOr(&g_flags, kFlagBadTarget);
    } else {
        wait_prerequisite_grid();
    }
    const auto count_of = [&](int e) -> long long {
        if constexpr (ALL)
            return hist[e];
        else
            return static_cast<long long>(__ldcg(&a.totals->counts[e]));
    };
    const int n = ALL ? s_n : static_cast<int>(__ldcg(&a.totals->n));
    const int bad = ALL ? s_bad : static_cast<int>(__ldcg(&a.totals->bad));
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e < a.E; e += NT)
            a.counts[e] = count_of(e);

    // the counts less their mean, (E f_e - sum) / E with the difference formed in
    // integers; then those of this lane's experts e = (j LPT + sub) VEC + v
    long long sum = 0;
    for (int e = threadIdx.x; e < a.E; e += NT)
        sum += count_of(e);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0)
        warp_sum64[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w)
        sum += warp_sum64[w];
    const float per_e = 1.f / static_cast<float>(a.E);
    const float fmean = static_cast<float>(sum) * per_e;
    for (int e = threadIdx.x; e < a.E; e += NT)
        centred[e] = static_cast<float>(count_of(e) * a.E - sum) * per_e;
    __syncthreads();
    float f[NJ * VEC];
#pragma unroll
    for (int i = 0; i < NJ * VEC; ++i) {
        const int e = (i / VEC * LPT + sub) * VEC + i % VEC;
        f[i] = e < a.E ? centred[e] : 0.f;
    }
    const float per_n = 1.f / static_cast<float>(n);
    const float ka = a.balance * static_cast<float>(a.E) / static_cast<float>(a.k) * per_n;  // a E / (k n)
    const float gscale = a.grad ? (a.grad_scale ? __ldg(a.grad_scale) : 1.f) * per_n : 0.f;
    const float ga = ka * gscale, gz = 2.f * a.z * gscale;
    const float la = ka * per_n, lz = a.z * per_n;  // of the loss: terms over n stay in range as long as their sum

    float part = 0.f, carry = 0.f;
    bool counted = t < a.T && mask[t];
    for (int64_t t0 = t - lane / LPT; t0 < a.T; t0 += groups) {  // one trip for the whole warp
        float x[NJ * VEC];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            if (counted && (j * LPT + sub) * VEC < a.E) {
                Unit::unpack(raw[j], x + j * VEC);
            } else {
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    x[j * VEC + v] = -INFINITY;
            }
        }
        const int64_t row = t;
        const bool in = row < a.T, live = counted;
        t += groups;
        load_row(t);
        counted = t < a.T && mask[t];

        float m = x[0];
#pragma unroll
        for (int i = 1; i < NJ * VEC; ++i)
            m = fmaxf(m, x[i]);
        m = group_max<LPT>(m);
        // about the maximum itself where its shift's rounding, 2^-24 of it in log2 units,
        // might outgrow exp2's range, or the shift fp32's (rows of a type's lowest value)
        const float far = fabsf(m) > kMoeFar && fabsf(m) < INFINITY ? m : 0.f;
        if (far != 0.f) {
#pragma unroll
            for (int i = 0; i < NJ * VEC; ++i)
                x[i] -= far;
            m = 0.f;
        }
        const float s = m == -INFINITY ? 0.f : shift_of(m);
        float d = 0.f, q = 0.f;
#pragma unroll
        for (int i = 0; i < NJ * VEC; ++i) {
            x[i] = exp2_shift(x[i], s);
            d += x[i];
            q = fmaf(x[i], f[i], q);
        }
        d = group_sum<LPT>(d);
        q = group_sum<LPT>(q);
        const float inv = 1.f / d, dot = q * inv;
        const float lse = far + fmaf(s, kLn2, logf(d));
        if (live && sub == 0) {
            const float v = fmaf(la, fmean + dot, lz * lse * lse);
            const float sum = part + v;
            carry += fabsf(part) >= fabsf(v) ? (part - sum) + v : (v - sum) + part;
            part = sum;
        }
        if (a.grad && in) {
            const float base = fmaf(-ga, dot, gz * lse);
            T *out = static_cast<T *>(a.grad) + row * a.gs;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int e = (j * LPT + sub) * VEC;
                if (e < a.E) {
                    float g[VEC];
#pragma unroll
                    for (int v = 0; v < VEC; ++v)
                        g[v] = live ? x[j * VEC + v] * inv * fmaf(ga, f[j * VEC + v], base) : 0.f;
                    Unit::store(out + e, g);
                }
            }
        }
    }
    if (!a.loss)
        return;

    // an infinite sum has no rounding errors to carry (inf - inf)
    double total = static_cast<double>(part) + (fabsf(part) < INFINITY ? static_cast<double>(carry) : 0.0);
    const auto add_up = [&]() {  // over the CTA, in thread 0
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            total += __shfl_xor_sync(0xffffffffu, total, off);
        __syncthreads();
        if (lane == 0)
            warp_part[threadIdx.x >> 5] = total;
        __syncthreads();
        if (threadIdx.x == 0) {
            total = 0.0;
            for (int w = 0; w < NT / 32; ++w)
                total += warp_part[w];
        }
    };
    add_up();
    if constexpr (!ALL) {
        if (threadIdx.x == 0) {
            a.part[blockIdx.x] = total;
            __threadfence();
            s_last = atomicAdd(&a.totals->done, 1u) == gridDim.x - 1;
        }
        __syncthreads();
        if (!s_last)
            return;
        __threadfence();
        total = 0.0;
        for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += NT)
            total += __ldcg(a.part + i);
        add_up();
    }
    if (threadIdx.x == 0)
        *a.loss = bad || n == 0 ? __int_as_float(0x7fc00000) : static_cast<float>(total);
}

}  // namespace gbce
