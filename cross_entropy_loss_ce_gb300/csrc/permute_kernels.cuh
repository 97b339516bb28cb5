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
// have a fixed order (j ascending) without atomics.  Measured (bf16, H 2048
// unless said, with 6.7 TB/s the rate of a plain copy):
//   dispatch  8192 x 4 tokens, 23% more rows by padding   29 us, 6.8 TB/s
//   combine   16384 x 8, H 4096                          177 us, 6.8 TB/s
//   its gradients  16384 x 8                             170 us, 6.7 TB/s
//   the plan  131072 x 8 slots of 256 experts             15 us in two kernels: the
//             time of a CTA's slots one after another, not of their 17 MB; 131072
//             slots 9 us, a single token 3 us
#pragma once

#include "row_kernels.cuh"

namespace gbce {

constexpr int kSortItems = 8;           // slots a thread holds
constexpr int kSortMaxExperts = 1024;
constexpr int kSortRoundBits = 13;      // a slot within a round of 1024 threads, beside 10 bits of expert
constexpr int kSortRankBits = 21;       // a rank within a CTA's slots, beside 10 bits of expert
constexpr int kPermuteThreads = 256;

struct SortArgs {
    const int64_t *experts;
    int64_t es;
    int64_t n;       // slots, T k
    int E, k, align;
    int64_t per_cta; // slots of a CTA, a multiple of its threads' kSortItems
    int rows;        // R
    void *table;     // slots of each CTA and expert: 16 bits, rows of sort_hist_stride(E), or 32 bits, rows of E
    bool one_round;  // a CTA ranks its slots at once
    int *position, *source, *offsets, *counts;
};

static_assert((1 << kSortRoundBits) == 1024 * kSortItems, "a round's slots");

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
        const int of_warp = lane < warps ? sums[lane] : 0;
        const int before = carry + __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0);
        const int all = __reduce_add_sync(0xffffffffu, of_warp);
        if (e < E)
            off[e] = before + sum - own;
        carry += all;
        __syncthreads();
    }
    if (threadIdx.x == 0)
        off[E] = carry;
    __syncthreads();
}

// Hands to visit(row) the rows of one expert that are no slot's, every 32nd from its `lane`-th on: its slots
// take `total` rows from `off` on, the next expert's begin at `next`.  Plans have up to 2^31 - 1 rows, so what is
// counted is the distance (below `align`): the row a step past the last may not be an int.
template <typename Visit>
__host__ __device__ __forceinline__ void sort_pad_rows(int off, int total, int next, int lane, const Visit &visit)
{
    const int first = off + total, pad = next - first;
    for (int i = lane; i < pad; i += 32)
        visit(first + i);
}

struct SortNoSlot {
    int *source;
    __host__ __device__ __forceinline__ void operator()(int row) const { source[row] = -1; }
};

// Rows that are no slot's: behind an expert's slots, and behind the last expert.
__device__ __forceinline__ void sort_fill(const SortArgs &a, const int *off, const int *total)
{
    const int lane = threadIdx.x & 31, warps = static_cast<int>(blockDim.x) >> 5;
    for (int e = static_cast<int>(blockIdx.x) * warps + static_cast<int>(threadIdx.x >> 5); a.align > 1 && e < a.E;
         e += static_cast<int>(gridDim.x) * warps)
        sort_pad_rows(off[e], total[e], off[e + 1], lane, SortNoSlot{a.source});
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
// consecutive slots at a time, lanes of the same expert find each other (each
// sets its bit in the warp's word of that expert; with a vote on each bit of the
// expert 131072 x 8 slots of 256 took 3 us more, with a match instruction 7) and
// count on from the warp's own histogram; the warps' histograms are then added up
// in order.  ALL: this CTA holds every slot and writes the plan; else expert and
// rank go to `position` (packed) and the CTA's counts to `table`.
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
    unsigned short *hist = chunk + hs;                                                     // [warps][hs]
    unsigned *bits = reinterpret_cast<unsigned *>(hist + warps * hs) + warp * a.E;         // [E] of each warp
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int e = threadIdx.x; e < a.E; e += static_cast<int>(blockDim.x))
        base[e] = 0;
    for (int e = lane; e < a.E; e += 32)
        bits[e] = 0;
    const int64_t first = blockIdx.x * a.per_cta;
    const int64_t last = first + a.per_cta < a.n ? first + a.per_cta : a.n;
    bool bad = false;
    if constexpr (ALL) {
        if (a.n == 0) {
            __syncthreads();
            sort_offsets(base, off, a.E, a.align, scan_sums);
        }
    }
    for (int64_t s0 = first; s0 < last; s0 += int64_t{blockDim.x} * kSortItems) {
        int expert[kSortItems], rank[kSortItems];
        const int64_t w0 = s0 + warp * (32 * kSortItems) + lane;
        int64_t id[kSortItems];  // all on their way before the first is looked at
        if (a.es == a.k) {
            const int64_t *p = a.experts + w0;
            const int left = static_cast<int>(last - w0 < 32 * kSortItems ? last - w0 : 32 * kSortItems);
#pragma unroll
            for (int i = 0; i < kSortItems; ++i)
                id[i] = i * 32 < left ? __ldg(p + i * 32) : -1;
        } else {
#pragma unroll
            for (int i = 0; i < kSortItems; ++i) {
                const int64_t s = w0 + i * 32;
                const unsigned t = static_cast<unsigned>(s) / static_cast<unsigned>(a.k);
                id[i] = s < last ? __ldg(a.experts + s + t * (a.es - a.k)) : -1;
            }
        }
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            bad |= id[i] < -1 || id[i] >= a.E;
            expert[i] = id[i] >= 0 && id[i] < a.E ? static_cast<int>(id[i]) : -1;
        }
        for (int i = threadIdx.x; i < warps * hs / 2; i += static_cast<int>(blockDim.x))
            reinterpret_cast<unsigned *>(hist)[i] = 0;
        __syncthreads();
        unsigned short *mine = hist + warp * hs;
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int e = expert[i];
            rank[i] = 0;
            if (s0 + warp * (32 * kSortItems) + i * 32 >= last)
                continue;  // nor has a later round
            if (e >= 0)
                atomicOr(bits + e, 1u << lane);
            __syncwarp();
            const unsigned peers = e >= 0 ? bits[e] : 0u, before = peers & ((1u << lane) - 1u);
            const int had = e >= 0 ? mine[e] : 0;
            rank[i] = had + __popc(before);
            __syncwarp();
            if (e >= 0 && !before) {  // the first of them counts them and clears the word
                mine[e] = static_cast<unsigned short>(had + __popc(peers));
                bits[e] = 0;
            }
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
    } else if (a.one_round) {  // counts of up to 8192, read two at a time
        unsigned short *counts = static_cast<unsigned short *>(a.table) + int64_t{blockIdx.x} * hs;
        for (int e = threadIdx.x; e < hs; e += static_cast<int>(blockDim.x))
            counts[e] = e < a.E ? static_cast<unsigned short>(base[e]) : 0;
    } else {
        int *counts = static_cast<int *>(a.table) + int64_t{blockIdx.x} * a.E;
        for (int e = threadIdx.x; e < a.E; e += static_cast<int>(blockDim.x))
            counts[e] = base[e];
    }
}

// The plan from the CTAs' counts: each CTA adds up what stands before it and
// places the slots of the CTA of its number, a round of them at a time, sorted
// in shared memory first: an expert's slots go to consecutive rows, so their
// stores go out together (one by one: 4 us more for 131072 x 8 slots).
// ONE: a.one_round.
template <bool ONE>
__global__ void __launch_bounds__(1024) sort_place_kernel(const SortArgs a)
{
    extern __shared__ int sort_smem[];
    __shared__ int scan_sums[32];
    const int threads = static_cast<int>(blockDim.x), cta = static_cast<int>(blockIdx.x);
    int *total = sort_smem;          // [E] slots of each expert
    int *before = total + a.E;       // [E] ... in earlier CTAs
    int *done = before + a.E;        // [E] ... in earlier rounds of this CTA
    int *mine = done + a.E;          // [E] ... in this round
    int *off = mine + a.E;           // [E + 1] the plan's offsets
    int *start = off + a.E + 1;      // [E + 1] the round's
    // [E] from a slot's rank among the CTA's of its expert to its row and to its place in the list
    int2 *to = reinterpret_cast<int2 *>(start + a.E + 1);
    int *list = reinterpret_cast<int *>(to + a.E);  // [slots of a round] by expert: expert and place in the round
    for (int e = threadIdx.x; e < 4 * a.E; e += threads)
        total[e] = 0;
    wait_prerequisite_grid();
    __syncthreads();
    // the first round's slots and the CTAs' counts are on their way together
    const int64_t first = cta * a.per_cta, round = int64_t{threads} * kSortItems;
    const int64_t last = first + a.per_cta < a.n ? first + a.per_cta : a.n;
    int packed[kSortItems];
    const auto load = [&](int64_t s0) {
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t s = s0 + i * threads + threadIdx.x;
            packed[i] = s < last ? __ldcg(a.position + s) : -1;
        }
    };
    load(first);
    // counts of a row: pairs of 16 bits, or single ones
    const int entries = ONE ? sort_hist_stride(a.E) / 2 : a.E;
    const int width = entries < threads ? entries : threads, groups = threads / width;
    const int group = static_cast<int>(threadIdx.x) / width, ctas = static_cast<int>(gridDim.x);
    for (int own = static_cast<int>(threadIdx.x) % width; group < groups && own < entries; own += width) {
        constexpr int kRows = ONE ? 16 : 32;
        int all[2] = {}, lower[2] = {};
        for (int b0 = group; b0 < ctas; b0 += kRows * groups) {
            unsigned c[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                c[i] = b0 + i * groups < ctas
                           ? __ldcg(static_cast<const unsigned *>(a.table) + int64_t{b0 + i * groups} * entries + own)
                           : 0u;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int n[2] = {static_cast<int>(ONE ? c[i] & 0xffffu : c[i]), static_cast<int>(ONE ? c[i] >> 16 : 0u)};
#pragma unroll
                for (int h = 0; h < (ONE ? 2 : 1); ++h) {
                    all[h] += n[h];
                    lower[h] += b0 + i * groups < cta ? n[h] : 0;
                    if (ONE && b0 + i * groups == cta && 2 * own + h < a.E)
                        mine[2 * own + h] = n[h];  // the round's
                }
            }
        }
#pragma unroll
        for (int h = 0; h < (ONE ? 2 : 1); ++h) {
            const int e = ONE ? 2 * own + h : own;
            if (e < a.E) {
                atomicAdd(total + e, all[h]);  // integers: any order, the same sum
                atomicAdd(before + e, lower[h]);
            }
        }
    }
    for (int64_t s0 = first; s0 < last; s0 += round) {
        if constexpr (!ONE) {
#pragma unroll
            for (int i = 0; i < kSortItems; ++i)
                if (packed[i] >= 0)
                    atomicAdd(mine + (packed[i] >> kSortRankBits), 1);
        }
        __syncthreads();
        if (s0 == first)
            sort_offsets(total, off, a.E, a.align, scan_sums);
        sort_offsets(mine, start, a.E, 1, scan_sums);
        for (int e = threadIdx.x; e < a.E; e += threads)
            to[e] = make_int2(off[e] + before[e], start[e] - done[e]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            if (packed[i] < 0)
                continue;
            const int e = packed[i] >> kSortRankBits, at = i * threads + static_cast<int>(threadIdx.x);
            const int rank = packed[i] & ((1 << kSortRankBits) - 1);
            const int2 by = to[e];
            a.position[s0 + at] = by.x + rank;
            list[by.y + rank] = e << kSortRoundBits | at;
        }
        if constexpr (!ONE)
            load(s0 + round);
        __syncthreads();
        for (int i = threadIdx.x; i < start[a.E]; i += threads) {
            const int2 by = to[list[i] >> kSortRoundBits];
            a.source[by.x - by.y + i] = static_cast<int>(s0) + (list[i] & ((1 << kSortRoundBits) - 1));
        }
        if (!ONE && s0 + round < last) {
            __syncthreads();
            for (int e = threadIdx.x; e < a.E; e += threads) {
                done[e] += mine[e];
                mine[e] = 0;
            }
            __syncthreads();
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
    int64_t zero_ctas;  // CTAs that zero the rows that are no slot's; those behind them take tokens
    int64_t token_ctas;
    bool weights_f32;   // else of the rows' type
};

// Zeroes the rows of `out` that are no slot's.  They lie in runs (behind an
// expert's slots, behind the last expert), so a warp looks at rows far apart.
template <typename Raw>
__device__ __forceinline__ void zero_rows(const PermuteArgs &a, int64_t os_units)
{
    const int lane = threadIdx.x & 31;
    const int64_t warps = a.zero_ctas * (blockDim.x >> 5);
    for (int64_t r0 = blockIdx.x * int64_t{blockDim.x >> 5} + (threadIdx.x >> 5); r0 < a.rows; r0 += warps * 32) {
        const int64_t r = r0 + lane * warps;
        unsigned todo = __ballot_sync(0xffffffffu, r < a.rows && __ldg(a.source + (r < a.rows ? r : 0)) < 0);
        while (todo) {
            const int i = __ffs(todo) - 1;
            todo &= todo - 1;
            Raw *row = static_cast<Raw *>(a.out) + (r0 + i * warps) * os_units;
            for (int u = lane; u < a.units; u += 32)
                row[u] = Raw{};
        }
    }
}

// x's rows to their places: bits are copied, so the type is that of a unit.  A
// warp takes 32 U units of a row; its stores need no waiting.  Bound by HBM.  Rows
// that are no slot's come first in the grid: 8192 x 4 x 2048 took 41 to 54 us with
// them as its tail on few SMs, and takes 29.
template <typename Raw, int U>
__global__ void __launch_bounds__(kPermuteThreads) dispatch_kernel(const PermuteArgs a, int64_t is_units, int64_t os_units)
{
    if (blockIdx.x < a.zero_ctas) {
        zero_rows<Raw>(a, os_units);
        return;
    }
    const int lane = threadIdx.x & 31;
    constexpr int kWarps = kPermuteThreads / 32;
    const int64_t all = a.T * a.segs;
    for (int64_t w = (blockIdx.x - a.zero_ctas) * int64_t{kWarps} + (threadIdx.x >> 5); w < all; w += a.token_ctas * kWarps) {
        const int64_t t = w / a.segs;
        const int u0 = static_cast<int>(w - t * a.segs) * (32 * U) + lane;
        const Raw *x = static_cast<const Raw *>(a.in) + t * is_units;
        Raw v[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            v[i] = u0 + i * 32 < a.units ? __ldcs(x + u0 + i * 32) : Raw{};
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

// VEC values of a row: 16 bytes, two 16-bit values, or one value.
template <typename T, int VEC>
struct RowUnit {
    static constexpr bool kPair = VEC == 2;
    using Raw = std::conditional_t<VEC == 1, T, std::conditional_t<kPair, unsigned, uint4>>;
    __device__ static __forceinline__ Raw load(const T *p)
    {
        if constexpr (VEC == 1)
            return *p;
        else
            return __ldcs(reinterpret_cast<const Raw *>(p));
    }
    __device__ static __forceinline__ void unpack(const Raw &r, float (&f)[VEC])
    {
        if constexpr (VEC == 1) {
            f[0] = Elem<T>::load(&r);
        } else if constexpr (kPair) {
            float v[8];
            Elem<T>::unpack(make_uint4(r, 0, 0, 0), v);
            f[0] = v[0];
            f[1] = v[1];
        } else {
            Elem<T>::unpack(r, f);
        }
    }
    __device__ static __forceinline__ void store(T *p, const float (&f)[VEC])
    {
        if constexpr (VEC == 1)
            Elem<T>::store(p, f[0]);
        else if constexpr (kPair)
            __stcs(reinterpret_cast<unsigned *>(p), Elem<T>::pack2(f[0], f[1]));
        else
            __stcs(reinterpret_cast<uint4 *>(p), Elem<T>::pack(f));
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

// KC rows of a token, U units of a lane each, are in flight together: 8 loads of
// 16 bytes a lane keep HBM busy with the 24 warps that 78 registers leave an SM.
// (The loads are predicated; as selects they went out two by two: 240 us for
// 177.)  A weight is applied in fp32 and the sum rounded once.
template <typename T, int VEC, int KC, int U>
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
        for (int j0 = 0; j0 < a.k; j0 += KC) {
            int p[KC];
            float wt[KC];
            typename Unit::Raw v[KC][U];
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                p[j] = j0 + j < a.k ? __ldg(a.position + t * a.k + j0 + j) : -1;
                wt[j] = j0 + j < a.k ? slot_weight<T>(a, t, j0 + j) : 0.f;
                if (p[j] >= a.rows)
                    p[j] = -1;
            }
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                const T *y = static_cast<const T *>(a.in) + p[j] * a.is;
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (p[j] >= 0 && u0 + i * 32 < a.units)
                        v[j][i] = Unit::load(y + int64_t{u0 + i * 32} * VEC);
            }
#pragma unroll
            for (int j = 0; j < KC; ++j) {
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

// combine's gradients: a token belongs to `segs` warps (1, 2, 4 or 8 of a CTA),
// which read its row of d_out once for up to KC slots, U units of a lane at a
// time, write that row times the weight to each slot's place and add up the
// products with each slot's y.  Stores are streaming ones; three CTAs an SM, though
// with 8 slots of 16-bit values that spills 4 to 108 bytes a thread (16384 x 8 x
// 2048 bf16: 170 us, with two and no spill 187; pairs, 2046: 224 and 216).
template <typename T, int VEC, int KC, int U>
__global__ void __launch_bounds__(kPermuteThreads, 3) combine_bwd_kernel(const PermuteArgs a)
{
    using Unit = RowUnit<T, VEC>;
    using Raw = typename Unit::Raw;
    constexpr int kWarps = kPermuteThreads / 32;
    __shared__ float part[kWarps][KC];
    if (blockIdx.x < a.zero_ctas) {
        zero_rows<Raw>(a, a.os / VEC);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int mine = warp / a.segs, first = (warp - mine * a.segs) * (32 * U) + lane;
    const int64_t tokens = kWarps / a.segs;  // of a CTA at a time
    for (int64_t t0 = (blockIdx.x - a.zero_ctas) * tokens; t0 < a.T; t0 += a.token_ctas * tokens) {
        const bool live = t0 + mine < a.T;  // else only there for the barriers
        if (!live && a.segs == 1)
            continue;
        const int64_t t = live ? t0 + mine : t0;
        const int units = live ? a.units : 0;
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
            for (int u = first; u < units; u += 32 * U * a.segs) {
                Raw gr[U], v[KC][U];
#pragma unroll
                for (int i = 0; i < U; ++i)
                    gr[i] = u + i * 32 < units ? Unit::load(g_row + int64_t{u + i * 32} * VEC) : Raw{};
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    const T *y = static_cast<const T *>(a.in) + p[j] * a.is;
#pragma unroll
                    for (int i = 0; i < U; ++i)
                        v[j][i] = a.d_weights && p[j] >= 0 && u + i * 32 < units
                                      ? Unit::load(y + int64_t{u + i * 32} * VEC)
                                      : Raw{};
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    float g[VEC];
                    Unit::unpack(gr[i], g);
#pragma unroll
                    for (int j = 0; j < KC; ++j) {
                        float f[VEC];
                        Unit::unpack(v[j][i], f);
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            dot[j] = fmaf(g[e], f[e], dot[j]);
                        if (a.out && p[j] >= 0 && u + i * 32 < units) {
#pragma unroll
                            for (int e = 0; e < VEC; ++e)
                                f[e] = wt[j] * g[e];
                            Unit::store(static_cast<T *>(a.out) + p[j] * a.os + int64_t{u + i * 32} * VEC, f);
                        }
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
                if (warp != mine * a.segs || !live)
                    continue;
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    dot[j] = 0.f;
                    for (int i = 0; i < a.segs; ++i)
                        dot[j] += part[warp + i][j];
                }
            }
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                if (lane != j || j0 + j >= a.k)
                    continue;
                const int64_t at = t * a.dws + j0 + j;
                const float d = p[j] < 0 ? 0.f : dot[j];  // not 0 times an infinity
                if (a.weights_f32)
                    static_cast<float *>(a.d_weights)[at] = d;
                else
                    Elem<T>::store(static_cast<T *>(a.d_weights) + at, d);
            }
        }
    }
}

}  // namespace gbce
