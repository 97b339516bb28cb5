// Host side of moe_sort, moe_dispatch, moe_combine and moe_combine_bwd:
// argument checks, launch shapes and the launches of permute_kernels.cuh.
// Part of gbce.cu.
#pragma once

#include "permute_kernels.cuh"

namespace gbce {
namespace {

constexpr int64_t kSortRound = 1024 * kSortItems;   // slots that one CTA ranks at once
constexpr int64_t kSortMaxPerCta = int64_t{1} << kSortRankBits;
constexpr int kMaxAlign = 1024;
constexpr int64_t kPermuteMaxCols = int64_t{1} << 24;
// with fewer warps a lane takes one unit, not several (304 tokens, 4 x 2048 bf16: combine 2.26 us with one and two
// units; 152: 1.96 and 2.26; 608: 2.98 and 2.78)
constexpr int64_t kPermuteWarpsPerSm = 16;

// Rows of a plan, or -1 where they pass 2^31 - 1.
int64_t plan_rows(int64_t T, int64_t E, int64_t k, int64_t align)
{
    const int64_t slots = T * k;
    const int64_t rows = round_up(slots + (E < slots ? E : slots) * (align - 1), align);
    return rows > INT32_MAX ? -1 : rows;
}

int check_plan(int64_t T, int64_t E, int64_t k, int64_t align)
{
    if (T < 0 || T > kMaxRows || E < 1 || E > kSortMaxExperts || k < 1 || k > kMoeMaxSlots || align < 1 ||
        align > kMaxAlign || T * k > INT32_MAX || plan_rows(T, E, k, align) < 0)
        return GBCE_ERR_SIZE;
    return GBCE_OK;
}

int sort_rank_smem(int E, int threads, bool all)
{
    const int warps = threads / 32;
    return (all ? 2 * E + 1 : E) * 4 + sort_hist_stride(E) * 2 * (warps + 1) + warps * E * 4;
}

int sort_place_smem(int E) { return (8 * E + 2 + static_cast<int>(kSortRound)) * 4; }

cudaError_t launch_sort(const Call &call, SortArgs a)
{
    cudaError_t e;
    if (a.n <= kSortRound) {
        const int threads = a.n <= 256 * kSortItems ? 256 : 1024;
        const int smem = sort_rank_smem(a.E, threads, true);
        a.per_cta = threads * kSortItems;
        if ((e = configure_smem(reinterpret_cast<const void *>(sort_rank_kernel<true>), call.device,
                                sort_rank_smem(kSortMaxExperts, 1024, true))) != cudaSuccess)
            return e;
        return launch_kernel(call, false, sort_rank_kernel<true>, 1, threads, smem, a);
    }
    // a CTA's time is one slot after another of its warps: small ones, while there are few (131072 slots of 256
    // experts: 9.2 us with 64 CTAs of 256 threads, 9.9 with 32 of 512, 14.9 with 16 of 1024); many CTAs make the sums
    // before each one long (262144: 9.9 us with 64 of 512, 18.2 with 128 of 256; 131072 x 8: 15.2 with 128 of 1024,
    // 17.9 with 512 threads, 39 with 256).  Between these sizes not always the best: 524288 take 14.9 with 64 of
    // 1024, 11.1 with 128 of 512
    int threads = 256;
    while (threads < 1024 && a.n > call.sms / 2 * threads * kSortItems)
        threads *= 2;
    const int64_t round = int64_t{threads} * kSortItems, rounds = (a.n + round - 1) / round;
    a.per_cta = (rounds + call.sms - 1) / call.sms * round;
    if (a.per_cta > kSortMaxPerCta)
        a.per_cta = kSortMaxPerCta;
    const int64_t ctas = (a.n + a.per_cta - 1) / a.per_cta;
    a.one_round = a.per_cta == round;
    const size_t row = a.one_round ? sort_hist_stride(a.E) * 2 : a.E * 4;
    PoolScratch scratch(call.stream);
    if ((e = scratch.get(call.device, static_cast<size_t>(ctas) * row)) != cudaSuccess)
        return e;
    a.table = scratch.p;
    e = configure_smem(reinterpret_cast<const void *>(sort_rank_kernel<false>), call.device,
                       sort_rank_smem(kSortMaxExperts, 1024, false));
    if (e == cudaSuccess)
        e = launch_kernel(call, false, sort_rank_kernel<false>, ctas, threads, sort_rank_smem(a.E, threads, false), a);
    void (*const place)(const SortArgs) = a.one_round ? sort_place_kernel<true> : sort_place_kernel<false>;
    if (e == cudaSuccess)
        e = configure_smem(reinterpret_cast<const void *>(place), call.device, sort_place_smem(kSortMaxExperts));
    if (e == cudaSuccess)
        e = launch_kernel(call, true, place, ctas, threads, sort_place_smem(a.E), a);
    return scratch.release(e);
}

// Do two of a plan's arrays, each from its first value to its last, share memory?  The second kernel follows what the
// first left in `position`, into shared memory too.
bool plan_arrays_overlap(const SortArgs &a)
{
    constexpr int64_t kMost = INT64_MAX / 16;  // of values: past any address
    const int64_t tokens = a.n / a.k, before = tokens > 0 && tokens - 1 <= kMost / a.es ? (tokens - 1) * a.es : kMost;
    const struct {
        const void *p;
        int64_t bytes;
    } arrays[] = {{a.experts, tokens > 0 ? (before + a.k) * 8 : 0},
                  {a.position, a.n * 4},
                  {a.source, int64_t{a.rows} * 4},
                  {a.offsets, (a.E + 1) * 4},
                  {a.counts, a.E * 4}};
    for (const auto &x : arrays)
        for (const auto &y : arrays) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(x.p), q = reinterpret_cast<uintptr_t>(y.p);
            if (&x != &y && x.bytes > 0 && y.bytes > 0 && p <= q && q - p < static_cast<uintptr_t>(x.bytes))
                return true;
        }
    return false;
}

int check_permute(int64_t T, int64_t H, int64_t k, int64_t rows, int dtype)
{
    const int st = check_common(T, H, dtype);
    if (st)
        return st;
    return H > kPermuteMaxCols || k < 1 || k > kMoeMaxSlots || T * k > INT32_MAX || rows < 0 || rows > INT32_MAX
               ? GBCE_ERR_SIZE
               : GBCE_OK;
}

// Rows of two matrices are made of whole units of `bytes`, and start on them.
bool in_units(size_t bytes, size_t es, int64_t H, const void *a, int64_t sa, const void *b, int64_t sb)
{
    const int64_t v = static_cast<int64_t>(bytes / es);
    return H % v == 0 && aligned_to(a, bytes) && sa % v == 0 && aligned_to(b, bytes) && sb % v == 0;
}

unsigned token_ctas(int64_t warps)
{
    const int64_t ctas = (warps + kPermuteThreads / 32 - 1) / (kPermuteThreads / 32);
    return static_cast<unsigned>(ctas < (1 << 30) ? ctas : (1 << 30));
}

// CTAs that look for rows that are no slot's, 256 of them at a time.
int64_t zero_ctas(const Call &call, int64_t rows)
{
    const int64_t ctas = (rows + kPermuteThreads - 1) / kPermuteThreads;
    return ctas < 2 * call.sms ? ctas : 2 * call.sms;
}

template <typename Raw, int U>
cudaError_t launch_dispatch_as(const Call &call, PermuteArgs a, size_t es)
{
    const int64_t v = static_cast<int64_t>(sizeof(Raw) / es);
    a.units = static_cast<int>(a.H / v);
    a.segs = (a.units + 32 * U - 1) / (32 * U);
    a.token_ctas = token_ctas(a.T * a.segs);
    a.zero_ctas = zero_ctas(call, a.rows);
    return launch_kernel(call, false, dispatch_kernel<Raw, U>, a.zero_ctas + a.token_ctas, kPermuteThreads, 0, a,
                         a.is / v, a.os / v);
}

cudaError_t launch_dispatch(const Call &call, const PermuteArgs &a)
{
    const size_t es = elem_size(call.dtype);
    if (in_units(16, es, a.H, a.in, a.is, a.out, a.os)) {
        // with stores enough behind each load one unit a lane is best (608 x 8 x 2048 bf16: 4.7 us, with four units
        // 6.3); a token's one or two copies need more loads in flight (1216 x 2 x 4096: 4.9 us with four, 5.6)
        const int64_t units = a.H * static_cast<int64_t>(es) / 16;
        return a.k > 2 || units <= 32 || a.T * ((units + 127) / 128) < kPermuteWarpsPerSm * call.sms
                   ? launch_dispatch_as<uint4, 1>(call, a, es)
                   : launch_dispatch_as<uint4, 4>(call, a, es);
    }
    if (in_units(4, es, a.H, a.in, a.is, a.out, a.os))
        return launch_dispatch_as<unsigned, 8>(call, a, es);
    return launch_dispatch_as<unsigned short, 8>(call, a, es);
}

template <typename T>
cudaError_t launch_combine(const Call &call, PermuteArgs a)
{
    constexpr int V = Elem<T>::kPerVec;
    const auto go = [&](void (*fn)(const PermuteArgs), int vec, int u) {
        a.units = static_cast<int>(a.H / vec);
        a.segs = (a.units + 32 * u - 1) / (32 * u);
        return launch_kernel(call, false, fn, token_ctas(a.T * a.segs), kPermuteThreads, 0, a);
    };
    if (!in_units(16, sizeof(T), a.H, a.in, a.is, a.out, a.os)) {
        // small units: many of a lane, or its loads are too few bytes (65536 x 2 x 2046 bf16: 201 us with 4 pairs, 144
        // with 16; 65536 x 2 x 2045: 391 with 4 values, 236 with 16; 32768 x 4 x 2045: 240 with 4, 172 with 8, 179
        // with 16); few where that leaves warps enough (33 x 4 x 2045: 2.1 us with 4 values, 2.9 with 16)
        const auto few = [&](int64_t units) {
            return a.T * ((units + 511) / 512) < kPermuteWarpsPerSm * call.sms;
        };
        if constexpr (sizeof(T) == 2)
            if (in_units(4, sizeof(T), a.H, a.in, a.is, a.out, a.os))
                return few(a.H / 2) ? go(combine_kernel<T, 2, 4, 4>, 2, 4) : go(combine_kernel<T, 2, 2, 16>, 2, 16);
        if (few(a.H))
            return go(combine_kernel<T, 1, 4, 4>, 1, 4);
        return a.k <= 2 ? go(combine_kernel<T, 1, 2, 16>, 1, 16) : go(combine_kernel<T, 1, 4, 8>, 1, 8);
    }
    // as many units of a lane as the row has, or as few as leave every SM its warps; twice as many where a
    // token has one or two rows (65536 x 2 x 2048 bf16: 148 us with two units, 133 with four)
    const int64_t units = a.H / V;
    if (units <= 32 || a.T * ((units + 63) / 64) < kPermuteWarpsPerSm * call.sms)
        return go(combine_kernel<T, V, 4, 1>, V, 1);
    if (a.k > 2 || units <= 64)
        return go(combine_kernel<T, V, 4, 2>, V, 2);
    return a.k == 1 ? go(combine_kernel<T, V, 1, 4>, V, 4) : go(combine_kernel<T, V, 2, 4>, V, 4);
}

template <typename T>
cudaError_t launch_combine_bwd(const Call &call, PermuteArgs a)
{
    constexpr int V = Elem<T>::kPerVec;
    const void *y = a.d_weights ? a.in : a.d_out;
    const int64_t y_stride = a.d_weights ? a.is : a.ds;
    const auto whole = [&](size_t bytes) {
        return in_units(bytes, sizeof(T), a.H, a.d_out, a.ds, y, y_stride) &&
               (!a.out || in_units(bytes, sizeof(T), a.H, a.out, a.os, a.out, a.os));
    };
    void (*fn)(const PermuteArgs) = nullptr;
    int vec = 1, u = a.k <= 4 ? 8 : 4;  // units of a lane
    if (whole(16)) {
        vec = V;
        u = a.k <= 2 ? 4 : (a.k <= 4 ? 2 : 1);
        fn = a.k <= 2 ? combine_bwd_kernel<T, V, 2, 4>
                      : (a.k <= 4 ? combine_bwd_kernel<T, V, 4, 2> : combine_bwd_kernel<T, V, 8, 1>);
    } else {
        fn = a.k <= 2 ? combine_bwd_kernel<T, 1, 2, 8>
                      : (a.k <= 4 ? combine_bwd_kernel<T, 1, 4, 8> : combine_bwd_kernel<T, 1, 8, 4>);
        if constexpr (sizeof(T) == 2)
            if (whole(4)) {
                vec = 2;
                fn = a.k <= 2 ? combine_bwd_kernel<T, 2, 2, 8>
                              : (a.k <= 4 ? combine_bwd_kernel<T, 2, 4, 8> : combine_bwd_kernel<T, 2, 8, 4>);
            }
    }
    // Warps of a token: each takes two trips or more over its part of the row (16384 x 8 x 2048 bf16: 172 us
    // with 4 warps, 193 with 8, 173 with one), one where tokens are too few to fill the SMs (152 x 8 x 4096: 5.5
    // us with 8 warps, 19 with one)
    a.units = static_cast<int>(a.H / vec);
    constexpr int kWarps = kPermuteThreads / 32;
    const int64_t trips = a.T < 2 * call.sms ? 1 : 2, spans = (a.H / vec + 32 * u - 1) / (32 * u);
    a.segs = 1;
    while (a.segs < kWarps && (trips == 1 ? a.segs < spans : 2 * a.segs * trips <= spans))
        a.segs *= 2;
    a.token_ctas = token_ctas(a.T * a.segs);
    a.zero_ctas = a.out ? zero_ctas(call, a.rows) : 0;
    return launch_kernel(call, false, fn, a.zero_ctas + a.token_ctas, kPermuteThreads, 0, a);
}

int check_weights(const void *w, int64_t stride, int wdtype, int64_t k, int dtype)
{
    if (!w)
        return GBCE_OK;
    if (wdtype != GBCE_F32 && wdtype != dtype)
        return GBCE_ERR_DTYPE;
    if (stride < k || stride > kMaxStride)
        return GBCE_ERR_SIZE;
    return aligned_to(w, elem_size(wdtype)) ? GBCE_OK : GBCE_ERR_ALIGN;
}

}  // namespace
}  // namespace gbce

extern "C" int64_t moe_plan_rows(int64_t T, int64_t E, int64_t k, int64_t align)
{
    return check_plan(T, E, k, align) ? -1 : plan_rows(T, E, k, align);
}

extern "C" int moe_sort(const int64_t *experts, int64_t experts_stride, int32_t *position, int32_t *source,
                        int32_t *offsets, int32_t *counts, int64_t T, int64_t E, int64_t k, int64_t align,
                        gbce_stream_t stream)
{
    const int st = check_plan(T, E, k, align);
    if (st)
        return st;
    if (experts_stride < k || experts_stride > kMaxStride)
        return GBCE_ERR_SIZE;
    if (!offsets || !counts || (T > 0 && (!experts || !position || !source)))
        return GBCE_ERR_NULL;
    if (!aligned_to(experts, 8) || !aligned_to(position, 4) || !aligned_to(source, 4) || !aligned_to(offsets, 4) ||
        !aligned_to(counts, 4))
        return GBCE_ERR_ALIGN;
    SortArgs a{};
    a.experts = experts;
    a.es = experts_stride;
    a.n = T * k;
    a.E = static_cast<int>(E);
    a.k = static_cast<int>(k);
    a.align = static_cast<int>(align);
    a.rows = static_cast<int>(plan_rows(T, E, k, align));
    a.position = position;
    a.source = source;
    a.offsets = offsets;
    a.counts = counts;
    if (plan_arrays_overlap(a))
        return GBCE_ERR_OVERLAP;
    Call call;
    const cudaError_t e = begin_call(&call, GBCE_F32, stream);
    if (e != cudaSuccess)
        return map_error(e);
    return map_error(launch_sort(call, a));
}

extern "C" int moe_dispatch(const void *x, int64_t x_stride, const int32_t *position, const int32_t *source,
                            void *out, int64_t out_stride, int64_t T, int64_t H, int64_t k, int64_t rows,
                            int dtype, gbce_stream_t stream)
{
    int st = check_permute(T, H, k, rows, dtype);
    if (st)
        return st;
    if ((T > 0 && !position) || (rows > 0 && !source))
        return GBCE_ERR_NULL;
    if ((st = check_matrix(x, x_stride, T, H, dtype)) || (st = check_matrix(out, out_stride, rows, H, dtype)))
        return st;
    if (!aligned_to(position, 4) || !aligned_to(source, 4))
        return GBCE_ERR_ALIGN;
    if (rows == 0)
        return GBCE_OK;
    Call call;
    const cudaError_t e = begin_call(&call, dtype, stream);
    if (e != cudaSuccess)
        return map_error(e);
    PermuteArgs a{};
    a.in = x;
    a.is = x_stride;
    a.out = out;
    a.os = out_stride;
    a.position = position;
    a.source = source;
    a.T = T;
    a.H = H;
    a.k = static_cast<int>(k);
    a.rows = static_cast<int>(rows);
    return map_error(launch_dispatch(call, a));
}

extern "C" int moe_combine(const void *y, int64_t y_stride, const int32_t *position, const void *weights,
                           int64_t weights_stride, int weights_dtype, void *out, int64_t out_stride, int64_t T,
                           int64_t H, int64_t k, int64_t rows, int dtype, gbce_stream_t stream)
{
    int st = check_permute(T, H, k, rows, dtype);
    if (st || (st = check_weights(weights, weights_stride, weights_dtype, k, dtype)))
        return st;
    if (T > 0 && !position)
        return GBCE_ERR_NULL;
    if ((st = check_matrix(y, y_stride, rows, H, dtype)) || (st = check_matrix(out, out_stride, T, H, dtype)))
        return st;
    if (!aligned_to(position, 4))
        return GBCE_ERR_ALIGN;
    if (T == 0)
        return GBCE_OK;
    Call call;
    const cudaError_t e = begin_call(&call, dtype, stream);
    if (e != cudaSuccess)
        return map_error(e);
    PermuteArgs a{};
    a.in = y;
    a.is = y_stride;
    a.out = out;
    a.os = out_stride;
    a.position = position;
    a.weights = weights;
    a.ws = weights_stride;
    a.weights_f32 = weights_dtype == GBCE_F32;
    a.T = T;
    a.H = H;
    a.k = static_cast<int>(k);
    a.rows = static_cast<int>(rows);
    switch (dtype) {
    case GBCE_F32: return map_error(launch_combine<float>(call, a));
    case GBCE_F16: return map_error(launch_combine<__half>(call, a));
    default: return map_error(launch_combine<__nv_bfloat16>(call, a));
    }
}

extern "C" int moe_combine_bwd(const void *d_out, int64_t d_out_stride, const void *y, int64_t y_stride,
                               const int32_t *position, const int32_t *source, const void *weights,
                               int64_t weights_stride, int weights_dtype, void *d_y, int64_t d_y_stride,
                               void *d_weights, int64_t d_weights_stride, int64_t T, int64_t H, int64_t k,
                               int64_t rows, int dtype, gbce_stream_t stream)
{
    int st = check_permute(T, H, k, rows, dtype);
    if (st || (st = check_weights(weights, weights_stride, weights_dtype, k, dtype)) ||
        (st = check_weights(d_weights, d_weights_stride, weights_dtype, k, dtype)))
        return st;
    if ((T > 0 && (!position || !weights)) || (d_y && rows > 0 && !source) || (!d_y && !d_weights && T > 0 && rows > 0))
        return GBCE_ERR_NULL;
    if ((st = check_matrix(d_out, d_out_stride, T, H, dtype)))
        return st;
    if (d_weights && (st = check_matrix(y, y_stride, rows, H, dtype)))
        return st;
    if (d_y && (st = check_matrix(d_y, d_y_stride, rows, H, dtype)))
        return st;
    if (!aligned_to(position, 4) || !aligned_to(source, 4))
        return GBCE_ERR_ALIGN;
    if (T == 0 && (!d_y || rows == 0))
        return GBCE_OK;
    Call call;
    const cudaError_t e = begin_call(&call, dtype, stream);
    if (e != cudaSuccess)
        return map_error(e);
    PermuteArgs a{};
    a.in = y;
    a.is = y_stride;
    a.out = rows > 0 ? d_y : nullptr;
    a.os = d_y_stride;
    a.d_out = d_out;
    a.ds = d_out_stride;
    a.position = position;
    a.source = source;
    a.weights = weights;
    a.ws = weights_stride;
    a.weights_f32 = weights_dtype == GBCE_F32;
    a.d_weights = d_weights;
    a.dws = d_weights_stride;
    a.T = T;
    a.H = H;
    a.k = static_cast<int>(k);
    a.rows = static_cast<int>(rows);
    switch (dtype) {
    case GBCE_F32: return map_error(launch_combine_bwd<float>(call, a));
    case GBCE_F16: return map_error(launch_combine_bwd<__half>(call, a));
    default: return map_error(launch_combine_bwd<__nv_bfloat16>(call, a));
    }
}
