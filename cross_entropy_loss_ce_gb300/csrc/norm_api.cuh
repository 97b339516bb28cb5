// Host side of grad_norm and clip_grad_norm: argument checks, the tables of
// tensors and the launches of norm_kernels.cuh.  Part of gbce.cu.
#pragma once

#include <algorithm>

#include "norm_kernels.cuh"

namespace gbce {
namespace {

constexpr int64_t kNormMaxTensors = int64_t{1} << 20;
constexpr int64_t kNormMaxValues = int64_t{1} << 40;  // of a tensor: 2^27 tiles
constexpr int64_t kNormMaxTiles = INT32_MAX / 2;      // of a launch, its grid's step included

struct TensorList {
    const void *const *in;
    void *const *out;  // NULL: not scaled
    const int64_t *values;
    const int *dtypes;
    int64_t n;
};

int check_tensors(const TensorList &l)
{
    if (l.n < 0 || l.n > kNormMaxTensors)
        return GBCE_ERR_SIZE;
    if (l.n > 0 && (!l.in || !l.values || !l.dtypes))
        return GBCE_ERR_NULL;
    for (int64_t i = 0; i < l.n; ++i) {
        if (!valid_dtype(l.dtypes[i]))
            return GBCE_ERR_DTYPE;
        if (l.values[i] < 0 || l.values[i] > kNormMaxValues)
            return GBCE_ERR_SIZE;
        if (l.values[i] > 0 && (!l.in[i] || (l.out && !l.out[i])))
            return GBCE_ERR_NULL;
        const size_t es = elem_size(l.dtypes[i]);
        if (!aligned_to(l.in[i], es) || (l.out && !aligned_to(l.out[i], es)))
            return GBCE_ERR_ALIGN;
    }
    return GBCE_OK;
}

// Does an output (the norm among them) share memory with another tensor, or with its own and starts elsewhere?
bool outputs_overlap(const TensorList &l, const float *norm)
{
    struct Span {
        uintptr_t first, last;
        bool out;
    };
    std::vector<Span> spans;
    spans.reserve(static_cast<size_t>(2 * l.n + 1));
    spans.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm) + sizeof(float), true});
    for (int64_t i = 0; i < l.n; ++i) {
        const size_t bytes = static_cast<size_t>(l.values[i]) * elem_size(l.dtypes[i]);
        const auto add = [&](const void *p, bool out) {
            const uintptr_t first = reinterpret_cast<uintptr_t>(p);
            spans.push_back({first, first + bytes, out});
        };
        if (!bytes)
            continue;
        add(l.out[i], true);
        if (l.in[i] != l.out[i])
            add(l.in[i], false);
    }
    std::sort(spans.begin(), spans.end(), [](const Span &a, const Span &b) { return a.first < b.first; });
    uintptr_t in_end = 0, out_end = 0;
    for (const Span &s : spans) {
        if (out_end > s.first || (s.out && in_end > s.first))
            return true;
        uintptr_t &end = s.out ? out_end : in_end;
        end = end > s.last ? end : s.last;
    }
    return false;
}

int64_t tensor_tiles(const void *p, int64_t values, int dtype)
{
    if (values == 0)
        return 0;
    const int64_t vecs = dtype == GBCE_F32 ? norm_geom<float>(p, values).vecs : norm_geom<__half>(p, values).vecs;
    return vecs > kNormTileVecs ? (vecs + kNormTileVecs - 1) / kNormTileVecs : 1;
}

// Fills a table from tensor i on, as far as it goes; returns the tensor it ends before.
template <int N>
int64_t fill_table(const TensorList &l, int64_t i, NormTable<N> *t)
{
    int64_t tiles = 0;
    int n = 0;
    for (; i < l.n && n < N; ++i) {
        const int64_t more = tensor_tiles(l.in[i], l.values[i], l.dtypes[i]);
        if (more == 0)
            continue;
        if (n > 0 && tiles + more > kNormMaxTiles)
            break;
        t->in[n] = static_cast<const char *>(l.in[i]);
        t->out[n] = l.out ? static_cast<char *>(l.out[i]) : nullptr;
        t->values[n] = l.values[i];
        t->type[n] = static_cast<unsigned char>(l.dtypes[i]);
        t->first[n++] = static_cast<int>(tiles);
        tiles += more;
    }
    t->first[n] = static_cast<int>(tiles);
    t->tensors = n;
    return i;
}

int64_t norm_grid(const Call &call, int64_t tiles)
{
    const int64_t most = call.sms * kNormCtasPerSm;
    return tiles < most ? tiles : most;
}

template <int KIND, int N>
cudaError_t launch_norm(const Call &call, const TensorList &l, float *norm, double max_norm, double eps, bool in_place)
{
    NormTable<N> t;
    int64_t next = fill_table<N>(l, 0, &t), parts = norm_grid(call, t.first[t.tensors]);
    const bool one = next == l.n;  // the only table is filled once
    while (next < l.n) {
        next = fill_table<N>(l, next, &t);
        parts += norm_grid(call, t.first[t.tensors]);
    }
    PoolScratch scratch(call.stream);
    cudaError_t e = scratch.get(call.device, static_cast<size_t>(parts + 1) * sizeof(double));
    if (e != cudaSuccess)
        return e;
    double *part = static_cast<double *>(scratch.p);
    int at = 0;
    const auto each = [&](auto launch) {  // launch(grid) for each table that holds a value
        for (int64_t i = 0; i < l.n && e == cudaSuccess;) {
            i = one ? l.n : fill_table<N>(l, i, &t);
            if (t.tensors > 0)
                e = launch(norm_grid(call, t.first[t.tensors]));
        }
    };
    each([&](int64_t grid) {
        double *here = part + at;
        const bool early = at > 0;
        at += static_cast<int>(grid);
        return launch_kernel(call, early, norm_parts_kernel<KIND, N>, grid, kNormThreads, 0, t, here);
    });
    float *result = norm;  // written by the first of the scaling kernels
    const double *total = part;
    int totals = at;
    const auto finish = [&](double *sum) {
        e = launch_kernel(call, at > 0, norm_finish_kernel<KIND>, 1, kNormThreads, 0, part, at, result, sum);
        result = nullptr;
    };
    if (e == cudaSuccess && l.out && !one && at > 0) {  // not by every CTA of every table's kernel
        finish(part + at);
        total = part + at;
        totals = 1;
    }
    if (l.out)
        each([&](int64_t grid) {
            float *here = result;
            result = nullptr;
            return launch_kernel(call, true, norm_scale_kernel<KIND, N>, grid, kNormThreads, 0, t, total, totals, here,
                                 max_norm, eps, in_place);
        });
    if (e == cudaSuccess && result)
        finish(nullptr);
    return scratch.release(e);
}

template <int N>
cudaError_t launch_norm_kind(const Call &call, const TensorList &l, int kind, float *norm, double max_norm, double eps,
                             bool in_place)
{
    switch (kind) {
    case GBCE_NORM_TWO: return launch_norm<kNormTwo, N>(call, l, norm, max_norm, eps, in_place);
    case GBCE_NORM_ONE: return launch_norm<kNormOne, N>(call, l, norm, max_norm, eps, in_place);
    default: return launch_norm<kNormMax, N>(call, l, norm, max_norm, eps, in_place);
    }
}

int norm_call(const TensorList &l, int kind, float *norm, double max_norm, double eps, gbce_stream_t stream)
{
    if (kind != GBCE_NORM_TWO && kind != GBCE_NORM_ONE && kind != GBCE_NORM_MAX)
        return GBCE_ERR_REDUCTION;
    if (!norm)
        return GBCE_ERR_NULL;
    const int st = check_tensors(l);
    if (st)
        return st;
    if (!aligned_to(norm, 4))
        return GBCE_ERR_ALIGN;
    bool in_place = true;
    for (int64_t i = 0; l.out && i < l.n; ++i)
        in_place &= l.in[i] == l.out[i] || l.values[i] == 0;
    try {
        if (l.out && outputs_overlap(l, norm))
            return GBCE_ERR_OVERLAP;
    } catch (...) {  // no memory on the host
        return GBCE_ERR_CUDA;
    }
    Call call;
    const cudaError_t e = begin_call(&call, GBCE_F32, stream);
    if (e != cudaSuccess)
        return map_error(e);
    return map_error(l.n <= kNormSmallTable ? launch_norm_kind<kNormSmallTable>(call, l, kind, norm, max_norm, eps, in_place)
                                            : launch_norm_kind<kNormTable>(call, l, kind, norm, max_norm, eps, in_place));
}

}  // namespace
}  // namespace gbce

extern "C" int grad_norm(const void *const *tensors, const int64_t *values, const int *dtypes, int64_t n, int kind,
                         float *norm, gbce_stream_t stream)
{
    return norm_call({tensors, nullptr, values, dtypes, n}, kind, norm, 0.0, 0.0, stream);
}

extern "C" int clip_grad_norm(const void *const *tensors, void *const *outs, const int64_t *values,
                              const int *dtypes, int64_t n, int kind, double max_norm, double eps, float *norm,
                              gbce_stream_t stream)
{
    if (n > 0 && !outs)
        return GBCE_ERR_NULL;
    if (!(max_norm >= 0.0) || !(eps >= 0.0))
        return GBCE_ERR_SIZE;
    return norm_call({tensors, n > 0 ? outs : nullptr, values, dtypes, n}, kind, norm, max_norm, eps, stream);
}
