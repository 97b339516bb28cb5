// Tokens sorted by expert and back: the plan of a router's choices (a stable
// counting sort of its slots), rows copied into that order, and rows brought
// back, weighted and summed, with the gradients of both.
//
// Slot s = t k + j holds the expert that token t goes to as its j-th.  With c_e
// the slots that hold e, o_0 = 0 and o_{e+1} = o_e + c_e rounded up to `align`,
//   position[s] = o_e + #{s' < s that hold e}   (-1 for a slot that holds none)
//   source[position[s]] = s                      (-1 for rows that are no slot's).
//   dispatch  out[position[t, j]] = x[t]
//   combine   out[t] = sum_j w[t, j] y[position[t, j]]
// Each is the other's gradient (w = 1); combine's with weights are
//   d_y[position[t, j]] = w[t, j] d_out[t],  d_w[t, j] = <d_out[t], y[position[t, j]]>.
//
// All of it is memory traffic.  Both directions go by tokens: dispatch reads a
// token's row once and writes it to its k places, combine reads the k rows
// and writes one, so every row crosses HBM once whatever the order, and sums
// have a fixed order (j ascending) without atomics.
#pragma once

#include "row_kernels.cuh"

namespace gbce {

constexpr int kSortItems = 8;           // slots a thread holds
constexpr int kSortMaxExperts = 1024;
constexpr int kSortRankBits = 21;       // a rank within a CTA's slots, beside 10 bits of expert
constexpr int kPermuteThreads = 256;

struct SortArgs {
    const int64_t *experts;
    int64_t es;
    int64_t n;       // slots, T k
    int E, k, align;
    int64_t per_cta; // slots of a CTA, a multiple of its threads' kSortItems
    int rows;        // R
    int *table;      // [gridDim.x, E] slots of each CTA and expert
    int *position, *source, *offsets, *counts;
};

__host__ __device__ __forceinline__ int sort_hist_stride(int E) { return (E + 1) / 2 * 2; }

// The offsets of segments v[e] rounded up to `align`, exclusive, in off[0 .. E]; all threads of the CTA.
__device__ __forceinline__ void sort_offsets(const int *v, int *off, int E, int align, int *sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += static_cast<int>(blockDim.x)) {
        const int e = e0 + static_cast<int>(threadIdx.x);
        const int own = e < E ? (v[e] + align - 1) / align * align : 0;
        int sum = own;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int up = __shfl_up_sync(0xffffffffu, sum, d);
            sum += lane >= d ? up : 0;
        }
        if (lane == 31)
            sums[warp] = sum;
        __syncthreads();
        int before = carry, all = 0;
        for (int w = 0; w < warps; ++w) {
            before += w < warp ? sums[w] : 0;
            all += sums[w];
        }
        if (e < E)
            off[e] = before + sum - own;
        carry += all;
        __syncthreads();
    }
    if (threadIdx.x == 0)
        off[E] = carry;
    __syncthreads();
}

// Rows that are no slot's: behind an expert's slots, and behind the last expert.
__device__ __forceinline__ void sort_fill(const SortArgs &a, const int *off, const int *total)
{
    for (int e = blockIdx.x; e < a.E; e += static_cast<int>(gridDim.x))
        for (int r = off[e] + total[e] + static_cast<int>(threadIdx.x); r < off[e + 1]; r += static_cast<int>(blockDim.x))
            a.source[r] = -1;
    for (int64_t r = off[a.E] + blockIdx.x * int64_t{blockDim.x} + threadIdx.x; r < a.rows;
         r += int64_t{gridDim.x} * blockDim.x)
        a.source[r] = -1;
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < a.E; e += static_cast<int>(blockDim.x))
            a.counts[e] = total[e];
        for (int e = threadIdx.x; e <= a.E; e += static_cast<int>(blockDim.x))
            a.offsets[e] = off[e];
    }
}

// Ranks the slots of a CTA by expert, in their order: a warp takes 32
// consecutive slots at a time, lanes of the same expert find each other with a
// match and count on from the warp's own histogram; the warps' histograms are
// then added up in order.  ALL: this CTA holds every slot and writes the plan;
// else expert and rank go to `position` (packed) and the CTA's counts to `table`.
template <bool ALL>
__global__ void __launch_bounds__(1024) sort_rank_kernel(const SortArgs a)
{
    extern __shared__ int sort_smem[];
    __shared__ int scan_sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int hs = sort_hist_stride(a.E);
    int *base = sort_smem;                  // [E] slots of earlier rounds; ALL: of all
    int *off = base + a.E;                  // [E + 1], ALL
    unsigned short *chunk = reinterpret_cast<unsigned short *>(off + (ALL ? a.E + 1 : 0));  // [E]
    unsigned short *hist = chunk + sort_hist_stride(a.E);                                  // [warps][hs]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int e = threadIdx.x; e < a.E; e += static_cast<int>(blockDim.x))
        base[e] = 0;
    const int64_t first = blockIdx.x * a.per_cta;
    const int64_t last = first + a.per_cta < a.n ? first + a.per_cta : a.n;
    bool bad = false;
    for (int64_t s0 = first; s0 < last; s0 += int64_t{blockDim.x} * kSortItems) {
        int expert[kSortItems], rank[kSortItems];
        const int64_t w0 = s0 + warp * (32 * kSortItems) + lane;
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t s = w0 + i * 32;
            int64_t e = -1;
            if (s < last) {
                if (a.es == a.k) {
                    e = __ldg(a.experts + s);
                } else {
                    const unsigned t = static_cast<unsigned>(s) / static_cast<unsigned>(a.k);
                    e = __ldg(a.experts + t * a.es + (s - int64_t{t} * a.k));
                }
                bad |= e < -1 || e >= a.E;
            }
            expert[i] = e >= 0 && e < a.E ? static_cast<int>(e) : -1;
        }
        for (int i = threadIdx.x; i < warps * hs / 2; i += static_cast<int>(blockDim.x))
            reinterpret_cast<unsigned *>(hist)[i] = 0;
        __syncthreads();
        unsigned short *mine = hist + warp * hs;
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int e = expert[i];
            const unsigned peers = __match_any_sync(0xffffffffu, e);
            const unsigned before = peers & ((1u << lane) - 1u);
            rank[i] = 0;
            if (e >= 0)
                rank[i] = mine[e] + __popc(before);
            __syncwarp();
            if (e >= 0 && !before)
                mine[e] = static_cast<unsigned short>(mine[e] + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += static_cast<int>(blockDim.x)) {
            unsigned sum = 0;
            for (int w = 0; w < warps; w += 8) {
                unsigned c[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    c[i] = w + i < warps ? hist[(w + i) * hs + e] : 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (w + i < warps)
                        hist[(w + i) * hs + e] = static_cast<unsigned short>(sum);
                    sum += c[i];
                }
            }
            chunk[e] = static_cast<unsigned short>(sum);
            if constexpr (ALL)
                base[e] = static_cast<int>(sum);
        }
        __syncthreads();
        if constexpr (ALL)
            sort_offsets(base, off, a.E, a.align, scan_sums);
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t s = w0 + i * 32;
            const int e = expert[i];
            if (s >= last)
                continue;
            if constexpr (ALL) {
                const int row = e < 0 ? -1 : off[e] + mine[e] + rank[i];
                a.position[s] = row;
                if (row >= 0)
                    a.source[row] = static_cast<int>(s);
            } else {
                a.position[s] = e < 0 ? -1 : (e << kSortRankBits) | (base[e] + mine[e] + rank[i]);
            }
        }
        if constexpr (!ALL) {
            __syncthreads();
            for (int e = threadIdx.x; e < a.E; e += static_cast<int>(blockDim.x))
                base[e] += chunk[e];
        }
    }
    if (bad)
        atomicOr(&g_flags, kFlagBadTarget);
    if constexpr (ALL) {
        sort_fill(a, off, base);
    } else {
        for (int e = threadIdx.x; e < a.E; e += static_cast<int>(blockDim.x))
            a.table[int64_t{blockIdx.x} * a.E + e] = base[e];
    }
}

// The plan from the CTAs' counts: each CTA adds up what stands before it and
// places the slots of the CTA of its number.
__global__ void __launch_bounds__(1024) sort_place_kernel(const SortArgs a)
{
    extern __shared__ int sort_smem[];
    __shared__ int scan_sums[32];
    int *total = sort_smem, *before = total + a.E, *off = before + a.E;  // [E], [E], [E + 1]
    for (int e = threadIdx.x; e < 2 * a.E; e += static_cast<int>(blockDim.x))
        total[e] = 0;
    wait_prerequisite_grid();
    __syncthreads();
    const int groups = static_cast<int>(blockDim.x) / a.E, ctas = static_cast<int>(gridDim.x);
    const int group = static_cast<int>(threadIdx.x) / a.E, e = static_cast<int>(threadIdx.x) % a.E;
    if (group < groups) {
        int all = 0, mine = 0;
#pragma unroll 8
        for (int b = group; b < ctas; b += groups) {
            const int c = __ldcg(a.table + int64_t{b} * a.E + e);
            all += c;
            mine += b < static_cast<int>(blockIdx.x) ? c : 0;
        }
        atomicAdd(total + e, all);  // integers: any order, the same sum
        atomicAdd(before + e, mine);
    }
    __syncthreads();
    sort_offsets(total, off, a.E, a.align, scan_sums);
    const int64_t first = blockIdx.x * a.per_cta;
    const int64_t last = first + a.per_cta < a.n ? first + a.per_cta : a.n;
    for (int64_t s0 = first + threadIdx.x; s0 < last; s0 += int64_t{blockDim.x} * kSortItems) {
        int packed[kSortItems];
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t s = s0 + i * int64_t{blockDim.x};
            packed[i] = s < last ? __ldcg(a.position + s) : -1;
        }
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t s = s0 + i * int64_t{blockDim.x};
            if (s < last && packed[i] >= 0) {
                const int x = packed[i] >> kSortRankBits;
                const int row = off[x] + before[x] + (packed[i] & ((1 << kSortRankBits) - 1));
                a.position[s] = row;
                a.source[row] = static_cast<int>(s);
            }
        }
    }
    sort_fill(a, off, total);
}

// ---------------------------------------------------------------------------

struct PermuteArgs {
    const void *in;     // dispatch: x [T, H]; combine: y [R, H]
    int64_t is;
    void *out;          // dispatch: [R, H]; combine: [T, H]; backward: d_y [R, H] or NULL
    int64_t os;
    const void *d_out;  // backward: [T, H]
    int64_t ds;
    const int *position, *source;
    const void *weights;  // [T, k] or NULL
    int64_t ws;
    void *d_weights;      // backward: [T, k] or NULL
    int64_t dws;
    int64_t T, H;
    int k, rows;
    int units;          // of a row: H in what a lane moves at a time
    int segs;           // warps that share a token's row
    int64_t token_ctas; // CTAs for tokens; those behind them zero the rows that are no slot's
    bool weights_f32;   // else of the rows' type
};

// Zeroes the rows of `out` that are no slot's, a warp 32 rows at a time.
template <typename Raw>
__device__ __forceinline__ void zero_rows(const PermuteArgs &a, int64_t os_units, int64_t cta, int64_t ctas)
{
    const int lane = threadIdx.x & 31;
    const int64_t warps = ctas * (blockDim.x >> 5);
    for (int64_t r0 = (cta * (blockDim.x >> 5) + (threadIdx.x >> 5)) * 32; r0 < a.rows; r0 += warps * 32) {
        const bool mine = r0 + lane < a.rows && __ldg(a.source + r0 + lane) < 0;
        unsigned todo = __ballot_sync(0xffffffffu, mine);
        while (todo) {
            const int i = __ffs(todo) - 1;
            todo &= todo - 1;
            Raw *row = static_cast<Raw *>(a.out) + (r0 + i) * os_units;
            for (int u = lane; u < a.units; u += 32)
                row[u] = Raw{};
        }
    }
}

// x's rows to their places: bits are copied, so the type is that of a unit.
template <typename Raw, int U>
__global__ void __launch_bounds__(kPermuteThreads) dispatch_kernel(const PermuteArgs a, int64_t is_units, int64_t os_units)
{
    if (static_cast<int64_t>(blockIdx.x) >= a.token_ctas) {
        zero_rows<Raw>(a, os_units, blockIdx.x - a.token_ctas, gridDim.x - a.token_ctas);
        return;
    }
    const int lane = threadIdx.x & 31;
    constexpr int kWarps = kPermuteThreads / 32;
    const int64_t all = a.T * a.segs;
    for (int64_t w = blockIdx.x * int64_t{kWarps} + (threadIdx.x >> 5); w < all; w += a.token_ctas * kWarps) {
        const int64_t t = w / a.segs;
        const int u0 = static_cast<int>(w - t * a.segs) * (32 * U) + lane;
        const Raw *x = static_cast<const Raw *>(a.in) + t * is_units;
        Raw v[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (u0 + i * 32 < a.units)
                v[i] = __ldcs(x + u0 + i * 32);
        const int *pos = a.position + t * a.k;
        for (int j0 = 0; j0 < a.k; j0 += 8) {
            int p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                p[j] = j0 + j < a.k ? __ldg(pos + j0 + j) : -1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (p[j] < 0 || p[j] >= a.rows)
                    continue;
                Raw *out = static_cast<Raw *>(a.out) + p[j] * os_units;
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (u0 + i * 32 < a.units)
                        out[u0 + i * 32] = v[i];
            }
        }
    }
}

// VEC values of a row: 16 bytes, or one value.
template <typename T, int VEC>
struct RowUnit {
    using Raw = std::conditional_t<VEC == 1, T, uint4>;
    __device__ static __forceinline__ Raw load(const T *p)
    {
        if constexpr (VEC == 1)
            return *p;
        else
            return __ldcs(reinterpret_cast<const uint4 *>(p));
    }
    __device__ static __forceinline__ void unpack(const Raw &r, float (&f)[VEC])
    {
        if constexpr (VEC == 1)
            f[0] = Elem<T>::load(&r);
        else
            Elem<T>::unpack(r, f);
    }
    __device__ static __forceinline__ void store(T *p, const float (&f)[VEC])
    {
        if constexpr (VEC == 1)
            Elem<T>::store(p, f[0]);
        else
            *reinterpret_cast<uint4 *>(p) = Elem<T>::pack(f);
    }
};

template <typename T>
__device__ __forceinline__ float slot_weight(const PermuteArgs &a, int64_t t, int j)
{
    if (!a.weights)
        return 1.f;
    if (a.weights_f32)
        return __ldg(static_cast<const float *>(a.weights) + t * a.ws + j);
    return Elem<T>::load(static_cast<const T *>(a.weights) + t * a.ws + j);
}

constexpr int kCombineSlots = 4;  // rows of a token whose loads are in flight together

template <typename T, int VEC, int U>
__global__ void __launch_bounds__(kPermuteThreads) combine_kernel(const PermuteArgs a)
{
    using Unit = RowUnit<T, VEC>;
    const int lane = threadIdx.x & 31;
    constexpr int kWarps = kPermuteThreads / 32;
    const int64_t all = a.T * a.segs;
    for (int64_t w = blockIdx.x * int64_t{kWarps} + (threadIdx.x >> 5); w < all; w += int64_t{gridDim.x} * kWarps) {
        const int64_t t = w / a.segs;
        const int u0 = static_cast<int>(w - t * a.segs) * (32 * U) + lane;
        float acc[U][VEC] = {};
        for (int j0 = 0; j0 < a.k; j0 += kCombineSlots) {
            int p[kCombineSlots];
            float wt[kCombineSlots];
            typename Unit::Raw v[kCombineSlots][U];
#pragma unroll
            for (int j = 0; j < kCombineSlots; ++j) {
                p[j] = j0 + j < a.k ? __ldg(a.position + t * a.k + j0 + j) : -1;
                wt[j] = j0 + j < a.k ? slot_weight<T>(a, t, j0 + j) : 0.f;
                if (p[j] >= a.rows)
                    p[j] = -1;
            }
#pragma unroll
            for (int j = 0; j < kCombineSlots; ++j) {
                const T *y = static_cast<const T *>(a.in) + p[j] * a.is;
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (p[j] >= 0 && u0 + i * 32 < a.units)
                        v[j][i] = Unit::load(y + int64_t{u0 + i * 32} * VEC);
            }
#pragma unroll
            for (int j = 0; j < kCombineSlots; ++j) {
                if (p[j] < 0)
                    continue;
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    float f[VEC];
                    Unit::unpack(v[j][i], f);
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        acc[i][e] = fmaf(wt[j], f[e], acc[i][e]);
                }
            }
        }
        T *out = static_cast<T *>(a.out) + t * a.os;
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (u0 + i * 32 < a.units)
                Unit::store(out + int64_t{u0 + i * 32} * VEC, acc[i]);
    }
}

// combine's gradients: a token belongs to `segs` warps (1, or all of a CTA),
// which read its row of d_out once for up to KC slots, write that row times
// the weight to each slot's place and add up the products with each slot's y.
template <typename T, int VEC, int KC>
__global__ void __launch_bounds__(kPermuteThreads) combine_bwd_kernel(const PermuteArgs a)
{
    using Unit = RowUnit<T, VEC>;
    constexpr int kWarps = kPermuteThreads / 32;
    __shared__ float part[kWarps][KC];
    if (static_cast<int64_t>(blockIdx.x) >= a.token_ctas) {
        if (a.out)
            zero_rows<typename Unit::Raw>(a, a.os / VEC, blockIdx.x - a.token_ctas, gridDim.x - a.token_ctas);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = a.segs == 1 ? 0 : warp, step = 32 * a.segs;
    const int64_t tokens = kWarps / a.segs;  // of a CTA at a time
    for (int64_t t0 = blockIdx.x * tokens; t0 < a.T; t0 += a.token_ctas * tokens) {
        const int64_t t = t0 + (a.segs == 1 ? warp : 0);
        if (t >= a.T)
            continue;  // segs == 1: nothing below waits for other warps
        const T *g_row = static_cast<const T *>(a.d_out) + t * a.ds;
        for (int j0 = 0; j0 < a.k; j0 += KC) {
            int p[KC];
            float wt[KC], dot[KC];
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                p[j] = j0 + j < a.k ? __ldg(a.position + t * a.k + j0 + j) : -1;
                wt[j] = j0 + j < a.k ? slot_weight<T>(a, t, j0 + j) : 0.f;
                dot[j] = 0.f;
                if (p[j] >= a.rows)
                    p[j] = -1;
            }
            for (int u = sub * 32 + lane; u < a.units; u += step) {
                typename Unit::Raw gr = Unit::load(g_row + int64_t{u} * VEC), v[KC];
                if (a.d_weights) {
#pragma unroll
                    for (int j = 0; j < KC; ++j)
                        if (p[j] >= 0)
                            v[j] = Unit::load(static_cast<const T *>(a.in) + p[j] * a.is + int64_t{u} * VEC);
                }
                float g[VEC];
                Unit::unpack(gr, g);
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    if (p[j] < 0)
                        continue;
                    if (a.out) {
                        float o[VEC];
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            o[e] = wt[j] * g[e];
                        Unit::store(static_cast<T *>(a.out) + p[j] * a.os + int64_t{u} * VEC, o);
                    }
                    if (a.d_weights) {
                        float f[VEC];
                        Unit::unpack(v[j], f);
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            dot[j] = fmaf(g[e], f[e], dot[j]);
                    }
                }
            }
            if (!a.d_weights)
                continue;
#pragma unroll
            for (int j = 0; j < KC; ++j)
                dot[j] = warp_sum(dot[j]);
            if (a.segs > 1) {
                __syncthreads();  // part of an earlier trip has been read
#pragma unroll
                for (int j = 0; j < KC; ++j)
                    if (lane == 0)
                        part[warp][j] = dot[j];
                __syncthreads();
                if (warp > 0)
                    continue;
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    dot[j] = 0.f;
                    for (int i = 0; i < kWarps; ++i)
                        dot[j] += part[i][j];
                }
            }
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                if (lane != j || j0 + j >= a.k)
                    continue;
                const int64_t at = t * a.dws + j0 + j;
                if (a.weights_f32)
                    static_cast<float *>(a.d_weights)[at] = dot[j];
                else
                    Elem<T>::store(static_cast<T *>(a.d_weights) + at, dot[j]);
            }
        }
    }
}

}  // namespace gbce
