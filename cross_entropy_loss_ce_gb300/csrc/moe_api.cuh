// Host side of moe_balance: argument checks, the choice of the rows kernel and
// the launches of moe_kernels.cuh.  Part of gbce.cu.
#pragma once

#include "moe_kernels.cuh"

namespace gbce {
namespace {

constexpr int64_t kMoeOneCtaSlots = 8192;   // slots up to which one CTA counts (no zeroing first)
constexpr int kMoeSmallThreads = 512;
constexpr int64_t kMoeRowsPerGroup = 2;   // rows that share a group's set-up, at least

using MoeFn = void (*)(const MoeArgs);

// Lanes that share a row of P = E / VEC units: about 16 values a lane, so that
// the reductions' shuffles are few and a warp holds several rows.
int moe_lanes(int P, int vec)
{
    if (vec == 1)
        return P <= 64 ? 16 : 32;
    return P <= 8 ? 4 : (P <= 32 ? 8 : (P <= 64 ? 16 : 32));
}

// The rows kernel for P units of VEC values a row.
template <typename T, int VEC, bool ALL, int NT>
MoeFn pick_moe_units(int P)
{
    if constexpr (VEC == 1) {
        if (P <= 16)
            return moe_rows_kernel<T, 1, 16, 1, ALL, NT>;
        if (P <= 64)
            return moe_rows_kernel<T, 1, 16, 4, ALL, NT>;
        if (P <= 128)
            return moe_rows_kernel<T, 1, 32, 4, ALL, NT>;
        if (P <= 512)
            return moe_rows_kernel<T, 1, 32, 16, ALL, NT>;
        return moe_rows_kernel<T, 1, 32, 32, ALL, NT>;
    } else {
        if (P <= 4)
            return moe_rows_kernel<T, VEC, 4, 1, ALL, NT>;
        if (P <= 8)
            return moe_rows_kernel<T, VEC, 4, 2, ALL, NT>;
        if (P <= 16)
            return moe_rows_kernel<T, VEC, 8, 2, ALL, NT>;
        if (P <= 32)
            return moe_rows_kernel<T, VEC, 8, 4, ALL, NT>;
        if (P <= 64)
            return moe_rows_kernel<T, VEC, 16, 4, ALL, NT>;
        if (VEC == 8 || P <= 128)
            return moe_rows_kernel<T, VEC, 32, 4, ALL, NT>;
        if constexpr (VEC == 4)
            return moe_rows_kernel<T, VEC, 32, 8, ALL, NT>;
    }
    return nullptr;  // not reached
}

template <typename T, bool ALL, int NT>
MoeFn pick_moe_vec(int vec, int E)
{
    if (vec == 1)
        return pick_moe_units<T, 1, ALL, NT>(E);
    if (vec == 4)
        return pick_moe_units<T, 4, ALL, NT>(E / 4);
    if constexpr (sizeof(T) == 2)
        return pick_moe_units<T, 8, ALL, NT>(E / 8);
    return nullptr;  // not reached: 4 fp32 values are 16 bytes
}

template <bool ALL, int NT>
MoeFn pick_moe(int dtype, int vec, int E)
{
    switch (dtype) {
    case GBCE_F32: return pick_moe_vec<float, ALL, NT>(vec, E);
    case GBCE_F16: return pick_moe_vec<__half, ALL, NT>(vec, E);
    default: return pick_moe_vec<__nv_bfloat16, ALL, NT>(vec, E);
    }
}

// Values a lane moves at a time: 16 bytes, 4 values, or one, whatever divides E
// and suits both matrices' rows.
int moe_vec(const MoeArgs &a, int dtype)
{
    const int64_t es = static_cast<int64_t>(elem_size(dtype));
    for (int64_t v = 16 / es; v >= 4; v /= 2) {
        const size_t bytes = static_cast<size_t>(v * es);
        if (a.E % v == 0 && aligned_to(a.logits, bytes) && (a.T <= 1 || a.ls % v == 0) &&
            (!a.grad || (aligned_to(a.grad, bytes) && (a.T <= 1 || a.gs % v == 0))))
            return static_cast<int>(v);
    }
    return 1;
}

struct MoeGrid {
    MoeFn fn;
    int device;
    int64_t ctas;
};
std::vector<MoeGrid> g_moe_grid;

// CTAs of a rows kernel that fit on the device at once (cached).
cudaError_t moe_resident(MoeFn fn, int device, int64_t sms, int64_t *out)
{
    std::lock_guard<std::mutex> lk(g_cfg_mu);
    for (const MoeGrid &g : g_moe_grid)
        if (g.fn == fn && g.device == device) {
            *out = g.ctas;
            return cudaSuccess;
        }
    RelaxedCapture relaxed;
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, kMoeThreads, 0);
    if (e != cudaSuccess)
        return e;
    *out = (n < 1 ? 1 : n) * sms;
    if (*out > kMoeMaxCtas)
        *out = kMoeMaxCtas;
    g_moe_grid.push_back({fn, device, *out});
    return cudaSuccess;
}

cudaError_t launch_moe(MoeArgs a, int dtype, int vec, void *scratch, int device, int64_t sms,
                       cudaStream_t stream)
{
    Carver place(scratch);
    a.totals = place.take<MoeTotals>(1);
    a.part = place.take<double>(kMoeMaxCtas);
    a.mask = place.take<unsigned char>(a.T);
    cudaError_t e;
    if (a.T * a.k <= kMoeOneCtaSlots) {
        moe_count_kernel<1024><<<1, 1024, 0, stream>>>(a);
    } else {
        if ((e = cudaMemsetAsync(a.totals, 0, sizeof(MoeTotals), stream)) != cudaSuccess)
            return e;
        const int64_t want = (a.T + kMoeThreads - 1) / kMoeThreads;
        moe_count_kernel<kMoeThreads><<<static_cast<unsigned>(want < 2 * sms ? want : 2 * sms), kMoeThreads,
                                        0, stream>>>(a);
    }
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    const MoeFn fn = pick_moe<false, kMoeThreads>(dtype, vec, a.E);
    const int lanes = moe_lanes(a.E / vec, vec);
    const int64_t rows = kMoeThreads / lanes * kMoeRowsPerGroup;  // of a CTA, at least
    const int64_t ctas = (a.T + rows - 1) / rows;
    int64_t most = 0;
    if ((e = moe_resident(fn, device, sms, &most)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas < most ? ctas : most), 1, 1);
    cfg.blockDim = dim3(kMoeThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<const MoeArgs>(a));
}

}  // namespace
}  // namespace gbce

extern "C" int moe_balance(const void *logits, int64_t logits_stride, const int64_t *experts,
                           int64_t experts_stride, int64_t *counts, float *loss, void *grad,
                           int64_t grad_stride, const float *grad_scale, int64_t T, int64_t E, int64_t k,
                           float balance_coef, float z_coef, int dtype, gbce_stream_t stream)
{
    int st = check_common(T, E, dtype);
    if (st)
        return st;
    if (E > kMoeMaxExperts || k < 1 || k > kMoeMaxSlots || experts_stride < k || experts_stride > kMaxStride)
        return GBCE_ERR_SIZE;
    if (!counts || (T > 0 && !experts) || (!loss && !grad))
        return GBCE_ERR_NULL;
    if ((st = check_matrix(logits, logits_stride, T, E, dtype)))
        return st;
    if (grad && (st = check_matrix(grad, grad_stride, T, E, dtype)))
        return st;
    if (!aligned_to(experts, 8) || !aligned_to(counts, 8) || !aligned_to(loss, 4) || !aligned_to(grad_scale, 4))
        return GBCE_ERR_ALIGN;
    Call call;
    cudaError_t e = begin_call(&call, dtype, stream);
    if (e != cudaSuccess)
        return map_error(e);
    MoeArgs a{};
    a.logits = logits;
    a.ls = logits_stride;
    a.experts = experts;
    a.es = experts_stride;
    a.T = T;
    a.E = static_cast<int>(E);
    a.k = static_cast<int>(k);
    a.counts = counts;
    a.loss = loss;
    a.grad = grad;
    a.gs = grad_stride;
    a.grad_scale = grad_scale;
    a.balance = balance_coef;
    a.z = z_coef;
    const int vec = moe_vec(a, dtype);
    if (T <= kMoeSmallTokens) {
        pick_moe<true, kMoeSmallThreads>(dtype, vec, a.E)<<<1, kMoeSmallThreads, 0, call.stream>>>(a);
        return map_error(cudaGetLastError());
    }
    PoolScratch scratch(call.stream);
    Carver size(nullptr);
    size.take<MoeTotals>(1);
    size.take<double>(kMoeMaxCtas);
    size.take<unsigned char>(T);
    if ((e = scratch.get(call.device, size.used)) != cudaSuccess)
        return map_error(e);
    return map_error(scratch.release(launch_moe(a, dtype, vec, scratch.p, call.device, call.sms, call.stream)));
}
