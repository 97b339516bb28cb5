// Host side of moe_balance: argument checks, the choice of the rows kernel and
// the launches of moe_kernels.cuh.  Part of gbce.cu.
#pragma once

#include "moe_kernels.cuh"

namespace gbce {
namespace {

constexpr int64_t kMoeSmallTokens = 256;  // tokens up to which one CTA does everything
constexpr int kMoeSmallThreads = 512;

using MoeFn = void (*)(const MoeArgs);

// The rows kernel for P = ceil(E / VEC) units of VEC values a row.
template <typename T, int VEC, bool ALL, int NT>
MoeFn pick_moe_units(int P)
{
    if (P <= 4)
        return moe_rows_kernel<T, VEC, 4, 1, ALL, NT>;
    if (P <= 16)
        return moe_rows_kernel<T, VEC, 16, 1, ALL, NT>;
    if (P <= 32)
        return moe_rows_kernel<T, VEC, 32, 1, ALL, NT>;
    if (P <= 64)
        return moe_rows_kernel<T, VEC, 32, 2, ALL, NT>;
    if (P <= 128)
        return moe_rows_kernel<T, VEC, 32, 4, ALL, NT>;
    if constexpr (VEC <= 4) {
        if (P <= 256)
            return moe_rows_kernel<T, VEC, 32, 8, ALL, NT>;
    }
    if constexpr (VEC == 1) {
        if (P <= 512)
            return moe_rows_kernel<T, VEC, 32, 16, ALL, NT>;
        return moe_rows_kernel<T, VEC, 32, 32, ALL, NT>;
    }
    return nullptr;  // not reached: P <= kMoeMaxExperts / VEC
}

template <bool ALL, int NT>
MoeFn pick_moe(int dtype, bool vec, int E)
{
    if (dtype == GBCE_F32)
        return vec ? pick_moe_units<float, 4, ALL, NT>(E / 4) : pick_moe_units<float, 1, ALL, NT>(E);
    if (dtype == GBCE_F16)
        return vec ? pick_moe_units<__half, 8, ALL, NT>(E / 8) : pick_moe_units<__half, 1, ALL, NT>(E);
    return vec ? pick_moe_units<__nv_bfloat16, 8, ALL, NT>(E / 8)
               : pick_moe_units<__nv_bfloat16, 1, ALL, NT>(E);
}

cudaError_t launch_moe(MoeArgs a, int dtype, bool vec, void *scratch, int device, int64_t sms,
                       cudaStream_t stream)
{
    if (a.T <= kMoeSmallTokens) {
        a.mask = static_cast<unsigned char *>(scratch);
        pick_moe<true, kMoeSmallThreads>(dtype, vec, a.E)<<<1, kMoeSmallThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    Carver place(scratch);
    a.totals = place.take<MoeTotals>(1);
    a.part = place.take<double>(kMoeMaxCtas);
    a.mask = place.take<unsigned char>(a.T);
    cudaError_t e = cudaMemsetAsync(a.totals, 0, sizeof(MoeTotals), stream);
    if (e != cudaSuccess)
        return e;
    const int64_t want = (a.T + kMoeThreads - 1) / kMoeThreads;
    moe_count_kernel<kMoeThreads><<<static_cast<unsigned>(want < 2 * sms ? want : 2 * sms), kMoeThreads,
                                    0, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    const MoeFn fn = pick_moe<false, kMoeThreads>(dtype, vec, a.E);
    const int units = vec ? a.E / static_cast<int>(16 / elem_size(dtype)) : a.E;
    const int lanes = units <= 4 ? 4 : (units <= 16 ? 16 : 32);
    const int64_t ctas = (a.T * lanes + kMoeThreads - 1) / kMoeThreads;
    const int64_t most = sms * 8 < kMoeMaxCtas ? sms * 8 : kMoeMaxCtas;
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
    const int64_t per = 16 / static_cast<int64_t>(elem_size(dtype));
    const bool vec = E % per == 0 && aligned_to(logits, 16) && (T <= 1 || logits_stride % per == 0) &&
                     (!grad || (aligned_to(grad, 16) && (T <= 1 || grad_stride % per == 0)));
    PoolScratch scratch(call.stream);
    const size_t bytes = sizeof(MoeTotals) + kMoeMaxCtas * sizeof(double) + static_cast<size_t>(T) + 1024;
    if ((e = scratch.get(call.device, bytes)) != cudaSuccess)
        return map_error(e);
    return map_error(scratch.release(launch_moe(a, dtype, vec, scratch.p, call.device, call.sms, call.stream)));
}
