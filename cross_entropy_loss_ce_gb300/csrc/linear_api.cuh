// Host side of the output-layer operators: argument checks, tensor maps, the
// scratch layout and the launches of linear_kernels.cuh.  Part of gbce.cu.
#pragma once

#include "linear_kernels.cuh"

namespace gbce {
namespace {

constexpr int64_t kGradPieceBytes = 512ll << 20;  // 16-bit logit gradients held at a time

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

std::atomic<EncodeTiled> g_encode{nullptr};

EncodeTiled encode_tiled()
{
    EncodeTiled fn = g_encode.load(std::memory_order_acquire);
    if (!fn) {
        RelaxedCapture relaxed;
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn = reinterpret_cast<EncodeTiled>(p);
        g_encode.store(fn, std::memory_order_release);
    }
    return fn;
}

// rows x cols 16-bit values, `stride` elements from row to row, read in boxes
// of 64 columns x `box_rows` rows with 128-byte swizzle; zeros outside.
cudaError_t make_map(CUtensorMap *map, const void *p, int dtype, int64_t rows, int64_t cols,
                     int64_t stride, int box_rows)
{
    const EncodeTiled fn = encode_tiled();
    if (!fn)
        return cudaErrorNotSupported;
    if (rows == 1)  // a single row may have any stride: give it a valid one
        stride = (cols + 7) / 8 * 8;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t step[2] = {1, 1};
    const CUresult r = fn(map, dtype == GBCE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          2, const_cast<void *>(p), dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// May a tensor map read this matrix as it stands?
bool mappable(const void *p, int64_t stride, int64_t rows)
{
    return aligned_to(p, 16) && (rows <= 1 || (stride % 8 == 0 && stride < (int64_t{1} << 38)));
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Consecutive 256-byte-aligned parts of one allocation; with a NULL base it
// only adds up their sizes.
struct Carver {
    char *base;
    size_t used = 0;
    explicit Carver(void *b) : base(static_cast<char *>(b)) {}
    template <typename T>
    T *take(int64_t count)
    {
        T *p = base ? reinterpret_cast<T *>(base + used) : nullptr;
        used += (static_cast<size_t>(count) * sizeof(T) + 255) / 256 * 256;
        return p;
    }
};

struct HeadScratch {
    int *n, *rows;      // divisor of the mean; listed rows
    unsigned *fail, *done;
    float *alpha;
    unsigned *arrived;
    int *idx, *tgt;
    float *l2, *rs, *gy, *xy;
    unsigned short *h;  // packed hidden states
    unsigned short *w;  // packed weights (rows a tensor map cannot read)
    float2 *part;
    float4 *best;
    unsigned short *g;
    float *acc, *slices, *runs;
};

struct HeadShape {
    int64_t M, K, V;
    int64_t kp;         // row stride of packed matrices: K rounded up to 128 bytes
    int64_t mp;         // rows of the packed hidden states
    bool skinny;
    bool pack_h, pack_w; // copies of the operands in scratch; a skinny forward without
                         // pack_h reads the hidden states as they stand
    int64_t parts;      // partial pairs of a row
    int64_t vp;         // backward: vocabulary rows of a piece
    int64_t pieces;
    int64_t slices;     // slices of split tiles, at most, of either gradient
    int grad_run, sum_run;  // backward: k-steps that tensor memory adds up at a time
    bool grad_runs, sum_runs;  // ... of a longer axis, with sums of earlier runs for run_pairs pairs
    int64_t run_pairs;
};

enum class HeadOp { Fwd, Bwd, Greedy };

HeadScratch carve(Carver &c, const HeadShape &s, HeadOp op, bool want_hidden)
{
    HeadScratch r{};
    int *words = c.take<int>(8);
    r.n = words;
    r.rows = words ? words + 1 : nullptr;
    r.fail = reinterpret_cast<unsigned *>(words ? words + 2 : nullptr);
    r.alpha = reinterpret_cast<float *>(words ? words + 3 : nullptr);
    r.done = reinterpret_cast<unsigned *>(words ? words + 4 : nullptr);
    if (op != HeadOp::Greedy) {
        r.idx = c.take<int>(s.M);
        r.tgt = c.take<int>(s.M);
    }
    if (s.pack_h)
        r.h = c.take<unsigned short>(s.mp * s.kp);
    if (s.pack_w)
        r.w = c.take<unsigned short>(s.V * s.kp);
    if (op == HeadOp::Bwd) {
        r.l2 = c.take<float>(s.M);
        r.rs = c.take<float>(s.M);
        r.gy = c.take<float>(s.M);
        r.g = c.take<unsigned short>(s.mp * s.vp);
        if (want_hidden && s.pieces > 1)
            r.acc = c.take<float>(s.mp * round_up(s.K, kPairN));
        r.arrived = c.take<unsigned>(kSplitCounters);
        r.slices = c.take<float>(2 * s.slices * kPairM * kPairN);
        if (s.run_pairs)
            r.runs = c.take<float>(s.run_pairs * kPairM * kPairN);
    } else {
        if (op == HeadOp::Fwd) {
            r.part = c.take<float2>(s.parts * s.mp);
            r.xy = c.take<float>(s.mp);
        } else {
            r.best = c.take<float4>(s.parts * s.mp);
        }
    }
    return r;
}

// Per-kernel one-time attributes (the dynamic shared memory it is launched with).
cudaError_t configure_smem(const void *fn, int device, int bytes)
{
    std::lock_guard<std::mutex> lk(g_cfg_mu);
    for (const FnConfig &c : g_cfg)
        if (c.fn == fn && c.device == device)
            return cudaSuccess;
    RelaxedCapture relaxed;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        g_cfg.push_back({fn, device});
    return e;
}

struct Call {
    int device;
    int64_t sms;
    cudaStream_t stream;
    int dtype;
};

// A kernel of a call.  All but the first may be set up while their predecessor
// on the stream still runs (`early`); they wait on the device before they touch
// anything.
template <typename... Args, typename... Given>
cudaError_t launch_kernel(const Call &call, bool early, void (*fn)(Args...), int64_t grid, int threads,
                          int smem, const Given &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = call.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<Args>(args)...);
}

template <Epi E, bool RUNS = false>
cudaError_t launch_pair(const Call &call, PairArgs a, const PairArgs &w, int64_t max_tiles,
                        bool early = true)
{
    a.drop_copy = g_drop_copy.load(std::memory_order_relaxed);
    using Fn = void (*)(const PairArgs, const PairArgs);
    const Fn fn = call.dtype == GBCE_BF16 ? static_cast<Fn>(pair_gemm_kernel<E, RUNS, __nv_bfloat16>)
                                          : static_cast<Fn>(pair_gemm_kernel<E, RUNS, __half>);
    const cudaError_t e = configure_smem(reinterpret_cast<const void *>(fn), call.device, kPairSmem);
    if (e != cudaSuccess)
        return e;
    const int64_t most = call.sms / 2 < kSplitUnits / 4 ? call.sms / 2 : kSplitUnits / 4;
    // split tiles use every pair they can
    const int64_t pairs = E == Epi::Both || max_tiles > most ? most : max_tiles;
    return launch_kernel(call, early, fn, 2 * pairs, kPairThreads, kPairSmem, a, w);
}

template <int NG, bool GREEDY>
cudaError_t launch_skinny_ng(const Call &call, SkinnyArgs a, int64_t ctas, bool early)
{
    a.drop_copy = g_drop_copy.load(std::memory_order_relaxed);
    const auto fn = skinny_kernel<NG, GREEDY>;
    const cudaError_t e =
        configure_smem(reinterpret_cast<const void *>(fn), call.device, skinny_smem<NG>());
    if (e != cudaSuccess)
        return e;
    return launch_kernel(call, early, fn, ctas, skinny_threads<NG>(), skinny_smem<NG>(), a);
}

int64_t gather_grid(const Call &call, int64_t rows)
{
    const int64_t want = (rows + 7) / 8, most = call.sms * 8;
    return want < most ? want : most;
}

// Lists the rows that count and packs them into g.dst (rows as far as s.mp).
template <bool BWD>
cudaError_t launch_start(const Call &call, const HeadShape &s, GatherArgs g, const PrepArgs &p)
{
    g.lds = s.kp;
    g.K = s.K;
    g.pad = static_cast<int>(s.skinny ? s.mp : kPairM);
    g.vec = mappable(g.src, g.ss, 2);
    g.wvec = g.vec && mappable(g.w, g.ws, 2);
    g.zvec = mappable(g.zero, g.zs, 2);
    const bool bf16 = call.dtype == GBCE_BF16;
    const int64_t grid = gather_grid(call, s.mp);
    if (p.M <= kStartRows)
        return launch_kernel(call, false, bf16 ? lin_start_kernel<__nv_bfloat16, BWD, 256> : lin_start_kernel<__half, BWD, 256>,
                             grid, 256, 0, g, p);
    const cudaError_t e = launch_kernel(call, false, lin_prep_kernel<1024, BWD>, 1, 1024, 0, p);
    if (e != cudaSuccess)
        return e;
    return launch_kernel(call, true, bf16 ? lin_gather_kernel<__nv_bfloat16, 256> : lin_gather_kernel<__half, 256>,
                         grid, 256, 0, g, p);
}

// Packed copy of n rows, and zeros up to a multiple of `pad`.  `first`: the first kernel of its call.
cudaError_t launch_pack(const Call &call, const HeadShape &s, const void *src, int64_t ss, void *dst,
                        int64_t n, int pad, bool first)
{
    GatherArgs g{};
    g.src = src;
    g.ss = ss;
    g.dst = dst;
    g.lds = s.kp;
    g.K = s.K;
    g.pad = pad;
    g.vec = mappable(src, ss, 2);
    return launch_kernel(call, !first, call.dtype == GBCE_BF16 ? lin_pack_kernel<__nv_bfloat16, 256> : lin_pack_kernel<__half, 256>,
                         gather_grid(call, round_up(n, pad)), 256, 0, g, n);
}

int check_head(const void *hidden, int64_t hs, const void *weight, int64_t ws, int64_t M, int64_t K,
               int64_t V, int dtype)
{
    if (dtype != GBCE_BF16 && dtype != GBCE_F16)
        return GBCE_ERR_DTYPE;
    // tiles of 256 x 256 are counted in 31 bits
    if (M < 0 || M > kMaxRows || K < 1 || K > (int64_t{1} << 24) || V < 1 || V > INT32_MAX - 1024 ||
        (round_up(M, 256) / 256 + kBand) * (round_up(V, 256) / 256) > INT32_MAX)
        return GBCE_ERR_SIZE;
    const int st = check_matrix(hidden, hs, M, K, dtype);
    return st ? st : check_matrix(weight, ws, V, K, dtype);
}

HeadShape head_shape(const Call &call, const void *hidden, int64_t hs, const void *weight, int64_t ws,
                     int64_t M, int64_t K, int64_t V, HeadOp op)
{
    HeadShape s{};
    s.M = M;
    s.K = K;
    s.V = V;
    s.kp = round_up(K, 64);
    s.skinny = op != HeadOp::Bwd && M <= kFewRows;
    s.mp = s.skinny ? (M <= 32 ? 32 : 64) : round_up(M, kPairM);
    // packed when rows are left out (any target may be ignore_index) or cannot be mapped
    s.pack_h = (op != HeadOp::Greedy && !s.skinny) || !mappable(hidden, hs, M);
    // weights whose rows start on 16 but not on 128 bytes are read as they are: a
    // copy to whole lines was measured (32000 classes, K 1000) and pays from about
    // 6000 rows on in the forward and 3000 in the backward, by at most 4% and 10%
    s.pack_w = !mappable(weight, ws, V);
    if (s.skinny) {
        const int64_t tiles = (V + 127) / 128;
        s.parts = tiles < call.sms ? tiles : call.sms;
    } else {
        s.parts = 2 * ((V + kPairN - 1) / kPairN);
    }
    if (op == HeadOp::Bwd) {
        int64_t vp = kGradPieceBytes / (s.mp * 2) / kPairN * kPairN;
        vp = vp < kPairN ? kPairN : vp;
        s.pieces = (V + vp - 1) / vp;
        s.vp = round_up((V + s.pieces - 1) / s.pieces, kPairN);
        s.pieces = (V + s.vp - 1) / s.vp;
        const int64_t rows = s.mp > s.vp ? s.mp : s.vp;
        const int64_t units = rows / kPairM * ((K + kPairN - 1) / kPairN) * kSplitMax;
        s.slices = units < kSplitUnits ? units : kSplitUnits;
        const int scale = call.dtype == GBCE_BF16 ? kBf16Runs : 1;
        s.grad_run = kGradRun * scale;
        s.sum_run = kSumRun * scale;
        s.grad_runs = K > s.grad_run * int64_t{kPairK};
        s.sum_runs = rows > s.sum_run * int64_t{kPairK};
        s.run_pairs = s.grad_runs || s.sum_runs ? call.sms / 2 : 0;
    }
    return s;
}

// The weights as the products read them: in place, or packed.
cudaError_t pack_weights(const Call &call, const HeadShape &s, const HeadScratch &r, const void *weight,
                         int64_t ws, const void **w, int64_t *wstride, bool first)
{
    *w = weight;
    *wstride = ws;
    if (!s.pack_w)
        return cudaSuccess;
    *w = r.w;
    *wstride = s.kp;
    return launch_pack(call, s, weight, ws, r.w, s.V, 1, first);
}

// Forward of `op` from prepared rows: the products and the merge.
template <bool GREEDY>
cudaError_t launch_head(const Call &call, const HeadShape &s, const HeadScratch &r, const void *h,
                        int64_t hstride, const void *w, int64_t wstride, int64_t hrows, MergeArgs m,
                        const PrepArgs *as_they_stand = nullptr)
{
    const bool early = s.pack_h || s.pack_w;  // not the call's first kernel
    cudaError_t e;
    const int kblocks = static_cast<int>((s.K + 63) / 64);
    m.part = r.part;
    m.best = r.best;
    m.parts = static_cast<int>(s.parts);
    m.n_ptr = GREEDY || as_they_stand ? nullptr : r.rows;
    m.n_host = static_cast<int>(s.M);
    m.idx = r.idx;
    m.xy = r.xy;
    if (s.skinny) {
        SkinnyArgs a{};
        if ((e = make_map(&a.w, w, call.dtype, s.V, s.K, wstride, 128)) != cudaSuccess ||
            (e = make_map(&a.h, h, call.dtype, hrows, s.K, hstride, static_cast<int>(s.mp))) != cudaSuccess)
            return e;
        a.n_ptr = m.n_ptr;
        a.n_host = m.n_host;
        a.kblocks = kblocks;
        a.V = s.V;
        a.tgt = r.tgt;
        a.targets = as_they_stand ? as_they_stand->targets : nullptr;
        a.part = r.part;
        a.best = r.best;
        a.ldp = s.parts;
        a.fail = GREEDY ? nullptr : r.fail;
        a.bf16 = call.dtype == GBCE_BF16;
        e = s.mp == 32 ? launch_skinny_ng<1, GREEDY>(call, a, s.parts, early)
                       : launch_skinny_ng<2, GREEDY>(call, a, s.parts, early);
    } else {
        PairArgs a{};
        if ((e = make_map(&a.a, h, call.dtype, hrows, s.K, hstride, 128)) != cudaSuccess ||
            (e = make_map(&a.b, w, call.dtype, s.V, s.K, wstride, 128)) != cudaSuccess)
            return e;
        a.n_ptr = m.n_ptr;
        a.n_host = m.n_host;
        a.tiles_n = static_cast<int>(s.parts / 2);
        a.kblocks = kblocks;
        a.fail = GREEDY ? nullptr : r.fail;
        a.part = r.part;
        a.best = r.best;
        a.ldp = s.parts;
        a.tgt = r.tgt;
        a.V = s.V;
        e = launch_pair<GREEDY ? Epi::Greedy : Epi::Stats>(call, a, a, s.mp / kPairM * a.tiles_n, early);
    }
    if (e != cudaSuccess)
        return e;
    m.h = h;
    m.hs = hstride;
    if (!m.w) {
        m.w = w;
        m.ws = wstride;
    }
    m.K = s.K;
    m.V = s.V;
    m.vec = mappable(h, hstride, hrows) && mappable(m.w, m.ws, s.V);
    if (!GREEDY && as_they_stand)
        return launch_kernel(call, true, call.dtype == GBCE_BF16 ? lin_few_kernel<__nv_bfloat16, 1024>
                                                                 : lin_few_kernel<__half, 1024>,
                             1, 1024, 0, m, *as_they_stand);
    if constexpr (!GREEDY)
        return launch_kernel(call, true, lin_merge_kernel<256>, (s.M + 7) / 8, 256, 0, m);
    else
        return launch_kernel(call, true, call.dtype == GBCE_BF16 ? lin_token_kernel<__nv_bfloat16, 128>
                                                         : lin_token_kernel<__half, 128>,
                           s.M, 128, 0, m);
}

cudaError_t launch_linear_fwd(const Call &call, const HeadShape &s, const HeadScratch &r,
                              const void *hidden, int64_t hs, const void *weight, int64_t ws,
                              const PrepArgs &prep)
{
    const bool few = s.skinny && !s.pack_h && s.M > 0;
    cudaError_t e = cudaSuccess;
    if (!few) {
        GatherArgs g{};
        g.src = hidden;
        g.ss = hs;
        g.dst = r.h;
        g.w = weight;
        g.ws = ws;
        g.xy = r.xy;
        e = launch_start<false>(call, s, g, prep);
        if (e != cudaSuccess || s.M == 0)
            return e;
    }
    const void *w;
    int64_t wstride;
    if ((e = pack_weights(call, s, r, weight, ws, &w, &wstride, few)) != cudaSuccess)
        return e;
    MergeArgs m{};
    m.row_loss = prep.row_loss;
    m.lse = prep.lse_out;
    m.loss = prep.reduction == GBCE_NONE ? nullptr : prep.loss;
    m.n_mean = r.n;
    m.fail = r.fail;
    m.done = r.done;
    m.M = s.M;
    m.reduction = prep.reduction;
    if (few) {  // lin_few_kernel reads the weights before it waits for their copy
        m.w = weight;
        m.ws = ws;
    }
    return few ? launch_head<false>(call, s, r, hidden, hs, w, wstride, s.M, m, &prep)
               : launch_head<false>(call, s, r, r.h, s.kp, w, wstride, s.mp, m);
}

cudaError_t launch_linear_bwd(const Call &call, const HeadShape &s, const HeadScratch &r,
                              const void *hidden, int64_t hs, const void *weight, int64_t ws,
                              const float *row_loss, void *d_hidden, int64_t dhs, void *d_weight,
                              int64_t dws, const PrepArgs &prep)
{
    GatherArgs g{};
    g.src = hidden;
    g.ss = hs;
    g.dst = r.h;
    g.w = row_loss ? nullptr : weight;
    g.ws = ws;
    g.gy = r.gy;
    g.row_loss = row_loss;
    g.zero = d_hidden;
    g.zs = dhs;
    g.M = s.M;
    g.V = s.V;
    g.ignore_index = prep.ignore_index;
    g.targets = prep.targets;
    cudaError_t e = launch_start<true>(call, s, g, prep);
    if (e != cudaSuccess)
        return e;
    const void *w;
    int64_t wstride;
    if ((e = pack_weights(call, s, r, weight, ws, &w, &wstride, false)) != cudaSuccess)
        return e;
    PairArgs grad{}, dw{}, dh{};
    const int tiles_k = static_cast<int>((s.K + kPairN - 1) / kPairN);
    if ((e = make_map(&grad.a, r.h, call.dtype, s.mp, s.K, s.kp, 128)) != cudaSuccess ||
        (e = make_map(&grad.b, w, call.dtype, s.V, s.K, wstride, 128)) != cudaSuccess ||
        (e = make_map(&dw.a, r.g, call.dtype, s.mp, s.vp, s.vp, 64)) != cudaSuccess ||
        (e = make_map(&dw.b, r.h, call.dtype, s.mp, s.K, s.kp, 64)) != cudaSuccess ||
        (e = make_map(&dh.a, r.g, call.dtype, s.mp, s.vp, s.vp, 128)) != cudaSuccess ||
        (e = make_map(&dh.b, w, call.dtype, s.V, s.K, wstride, 64)) != cudaSuccess)
        return e;
    for (PairArgs *a : {&grad, &dw, &dh}) {
        a->n_ptr = r.rows;
        a->fail = r.fail;
        a->alpha = r.alpha;
        a->idx = r.idx;
        a->tgt = r.tgt;
        a->l2 = r.l2;
        a->rs = r.rs;
        a->gy = r.gy;
        a->g = r.g;
        a->ldg = s.vp;
        a->cols = s.K;
        a->acc = r.acc;
        a->slices = r.slices;
        a->arrived = r.arrived;
        a->run = a == &grad ? s.grad_run : s.sum_run;
        a->runs = r.runs;
    }
    grad.kblocks = static_cast<int>((s.K + 63) / 64);
    dw.tiles_n = d_weight ? tiles_k : 0;  // none: no tiles
    dh.tiles_n = d_hidden ? tiles_k : 0;
    dw.slices = r.slices + s.slices * kPairM * kPairN;
    dw.arrived = r.arrived + kSplitUnits / 2 * 16;
    dw.ldo = dws;
    dw.vec = aligned_to(d_weight, 16) && dws % 8 == 0;
    dh.out = d_hidden;
    dh.ldo = dhs;
    dh.vec = aligned_to(d_hidden, 16) && dhs % 8 == 0;
    for (int64_t p = 0; p < s.pieces; ++p) {
        const int64_t v0 = p * s.vp;
        const int64_t vn = s.V - v0 < s.vp ? s.V - v0 : s.vp;
        const int tiles_v = static_cast<int>((vn + kPairN - 1) / kPairN);
        grad.b_row0 = dh.b_row0 = static_cast<int>(v0);
        grad.V = vn;
        grad.tiles_n = tiles_v;
        const int64_t tiles = s.mp / kPairM * tiles_v;
        if ((e = s.grad_runs ? launch_pair<Epi::Grad, true>(call, grad, grad, tiles)
                             : launch_pair<Epi::Grad>(call, grad, grad, tiles)) != cudaSuccess)
            return e;
        if (d_weight) {
            dw.out = static_cast<unsigned short *>(d_weight) + v0 * dws;
            dw.rows = vn;
            dw.tiles_m = tiles_v;
        }
        dh.kblocks = tiles_v * (kPairN / kPairK);  // G holds zeros up to whole tiles
        dh.first = p == 0;
        dh.last = p == s.pieces - 1;
        if ((e = s.sum_runs ? launch_pair<Epi::Both, true>(call, dh, dw, 0)
                            : launch_pair<Epi::Both>(call, dh, dw, 0)) != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

// The pool of the current device and one allocation from it, freed on the
// stream when the call's launches are queued.
struct PoolScratch {
    void *p = nullptr;
    cudaStream_t stream;
    explicit PoolScratch(cudaStream_t s) : stream(s) {}
    cudaError_t get(int device, size_t bytes)
    {
        cudaMemPool_t pool;
        cudaError_t e = pool_for(device, &pool);
        if (e == cudaSuccess && (e = cudaMallocFromPoolAsync(&p, bytes, pool, stream)) != cudaSuccess) {
            p = nullptr;
            cudaGetLastError();  // reported here: a later launch must not find it
        }
        return e;
    }
    cudaError_t release(cudaError_t e)
    {
        const cudaError_t ef = p ? cudaFreeAsync(p, stream) : cudaSuccess;
        p = nullptr;
        return e != cudaSuccess ? e : ef;
    }
};

cudaError_t begin_call(Call *call, int dtype, gbce_stream_t stream)
{
    call->dtype = dtype;
    call->stream = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = cudaGetDevice(&call->device);
    if (e != cudaSuccess)
        return e;
    call->sms = current_sm_count();
    return call->sms < 2 ? cudaErrorInvalidDevice : cudaSuccess;
}

}  // namespace
}  // namespace gbce

extern "C" int linear_ce_fwd(const void *hidden, int64_t hidden_stride, const void *weight,
                             int64_t weight_stride, const int64_t *targets, float *loss,
                             float *row_loss, float *lse, int64_t M, int64_t K, int64_t V,
                             int64_t ignore_index, int dtype, int reduction, gbce_stream_t stream)
{
    int st = check_head(hidden, hidden_stride, weight, weight_stride, M, K, V, dtype);
    if (st)
        return st;
    if (reduction != GBCE_MEAN && reduction != GBCE_SUM && reduction != GBCE_NONE)
        return GBCE_ERR_REDUCTION;
    if ((reduction != GBCE_NONE && !loss) || (M > 0 && (!targets || !row_loss)))
        return GBCE_ERR_NULL;
    if (!aligned_to(targets, 8) || !aligned_to(loss, 4) || !aligned_to(row_loss, 16) || !aligned_to(lse, 4))
        return GBCE_ERR_ALIGN;
    Call call;
    cudaError_t e = begin_call(&call, dtype, stream);
    if (e != cudaSuccess)
        return map_error(e);
    const HeadShape s = head_shape(call, hidden, hidden_stride, weight, weight_stride, M, K, V, HeadOp::Fwd);
    Carver size(nullptr);
    carve(size, s, HeadOp::Fwd, false);
    PoolScratch scratch(call.stream);
    if ((e = scratch.get(call.device, size.used)) != cudaSuccess)
        return map_error(e);
    Carver place(scratch.p);
    const HeadScratch r = carve(place, s, HeadOp::Fwd, false);
    PrepArgs prep{};
    prep.targets = targets;
    prep.M = M;
    prep.V = V;
    prep.ignore_index = ignore_index;
    prep.n_out = r.n;
    prep.rows_out = r.rows;
    prep.fail = r.fail;
    prep.done = r.done;
    prep.idx = r.idx;
    prep.tgt = r.tgt;
    prep.reduction = reduction;
    prep.loss = loss;
    prep.row_loss = row_loss;
    prep.lse_out = lse;
    return map_error(scratch.release(
        launch_linear_fwd(call, s, r, hidden, hidden_stride, weight, weight_stride, prep)));
}

extern "C" int linear_ce_bwd(const void *hidden, int64_t hidden_stride, const void *weight,
                             int64_t weight_stride, const int64_t *targets, const float *lse,
                             const float *grad_scale, void *d_hidden, int64_t d_hidden_stride,
                             void *d_weight, int64_t d_weight_stride, int64_t M, int64_t K, int64_t V,
                             int64_t ignore_index, int dtype, int reduction, gbce_stream_t stream)
{
    return linear_ce_bwd_ex(hidden, hidden_stride, weight, weight_stride, targets, lse, nullptr, grad_scale,
                            d_hidden, d_hidden_stride, d_weight, d_weight_stride, M, K, V, ignore_index, dtype,
                            reduction, stream);
}

extern "C" int linear_ce_bwd_ex(const void *hidden, int64_t hidden_stride, const void *weight,
                                int64_t weight_stride, const int64_t *targets, const float *lse,
                                const float *row_loss, const float *grad_scale, void *d_hidden,
                                int64_t d_hidden_stride, void *d_weight, int64_t d_weight_stride, int64_t M,
                                int64_t K, int64_t V, int64_t ignore_index, int dtype, int reduction,
                                gbce_stream_t stream)
{
    int st = check_head(hidden, hidden_stride, weight, weight_stride, M, K, V, dtype);
    if (st)
        return st;
    if (reduction != GBCE_MEAN && reduction != GBCE_SUM && reduction != GBCE_NONE)
        return GBCE_ERR_REDUCTION;
    if ((!d_hidden && !d_weight && M > 0) || (M > 0 && (!targets || !lse)))
        return GBCE_ERR_NULL;
    if (d_hidden && (st = check_matrix(d_hidden, d_hidden_stride, M, K, dtype)))
        return st;
    if (d_weight && (st = check_matrix(d_weight, d_weight_stride, V, K, dtype)))
        return st;
    if (!aligned_to(targets, 8) || !aligned_to(lse, 4) || !aligned_to(row_loss, 4) || !aligned_to(grad_scale, 4))
        return GBCE_ERR_ALIGN;
    if (M == 0 && !d_weight)
        return GBCE_OK;
    Call call;
    cudaError_t e = begin_call(&call, dtype, stream);
    if (e != cudaSuccess)
        return map_error(e);
    // M == 0 leaves the weights' gradient: zeros, by the same path with no row listed
    const HeadShape s = head_shape(call, hidden, hidden_stride, weight, weight_stride, M > 0 ? M : 1, K, V, HeadOp::Bwd);
    Carver size(nullptr);
    carve(size, s, HeadOp::Bwd, d_hidden != nullptr);
    PoolScratch scratch(call.stream);
    if ((e = scratch.get(call.device, size.used)) != cudaSuccess)
        return map_error(e);
    Carver place(scratch.p);
    const HeadScratch r = carve(place, s, HeadOp::Bwd, d_hidden != nullptr);
    PrepArgs prep{};
    prep.targets = targets;
    prep.M = M;
    prep.V = V;
    prep.ignore_index = ignore_index;
    prep.n_out = r.n;
    prep.rows_out = r.rows;
    prep.fail = r.fail;
    prep.done = r.done;
    prep.idx = r.idx;
    prep.tgt = r.tgt;
    prep.reduction = reduction;
    prep.lse_in = lse;
    prep.grad_scale = grad_scale;
    prep.l2 = r.l2;
    prep.rs = r.rs;
    prep.alpha = r.alpha;
    prep.arrived = r.arrived;
    prep.head = dtype == GBCE_F16 ? 16384.f : 2.f;
    return map_error(scratch.release(launch_linear_bwd(call, s, r, hidden, hidden_stride, weight,
                                                       weight_stride, row_loss, M > 0 ? d_hidden : nullptr,
                                                       d_hidden_stride, d_weight, d_weight_stride, prep)));
}

extern "C" int linear_greedy(const void *hidden, int64_t hidden_stride, const void *weight,
                             int64_t weight_stride, int64_t *tokens, float *logprob, int64_t M,
                             int64_t K, int64_t V, int dtype, gbce_stream_t stream)
{
    int st = check_head(hidden, hidden_stride, weight, weight_stride, M, K, V, dtype);
    if (st)
        return st;
    if (M > 0 && (!tokens || !logprob))
        return GBCE_ERR_NULL;
    if (!aligned_to(tokens, 8) || !aligned_to(logprob, 4))
        return GBCE_ERR_ALIGN;
    if (M == 0)
        return GBCE_OK;
    Call call;
    cudaError_t e = begin_call(&call, dtype, stream);
    if (e != cudaSuccess)
        return map_error(e);
    const HeadShape s = head_shape(call, hidden, hidden_stride, weight, weight_stride, M, K, V, HeadOp::Greedy);
    Carver size(nullptr);
    carve(size, s, HeadOp::Greedy, false);
    PoolScratch scratch(call.stream);
    if ((e = scratch.get(call.device, size.used)) != cudaSuccess)
        return map_error(e);
    Carver place(scratch.p);
    const HeadScratch r = carve(place, s, HeadOp::Greedy, false);
    const void *w = weight, *h = hidden;
    int64_t wstride = weight_stride, hstride = hidden_stride, hrows = M;
    if (s.pack_h) {
        e = launch_pack(call, s, hidden, hidden_stride, r.h, M, static_cast<int>(s.skinny ? s.mp : kPairM), true);
        h = r.h;
        hstride = s.kp;
        hrows = s.mp;
    }
    if (e == cudaSuccess)
        e = pack_weights(call, s, r, weight, weight_stride, &w, &wstride, !s.pack_h);
    if (e == cudaSuccess) {
        MergeArgs m{};
        m.token = tokens;
        m.logprob = logprob;
        e = launch_head<true>(call, s, r, h, hstride, w, wstride, hrows, m);
    }
    return map_error(scratch.release(e));
}
