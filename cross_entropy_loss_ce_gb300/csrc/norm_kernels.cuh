// The norm of many tensors taken as one vector, and the tensors scaled so that
// it keeps a limit:
//   n = (sum g^2)^(1/2), sum |g| or max |g|
//   out = f g,  f = min(1, max_norm / (n + eps))
//
// The factor needs every value before the first result, so the clipped form
// reads twice and writes once; tensors that fit in L2 come from HBM once.  The
// tensors are cut into tiles of 32 KB and a grid of the device's size takes
// them in turn, whatever tensor they are of; a tensor below that costs a tile.
// The table of up to 1024 tensors travels in the kernel's parameters, so a call
// copies nothing to the device and can be captured; a longer list takes a launch
// for each 1024, twice when it is clipped.
// Both passes are bound by HBM: 1.3e9 values of bf16 (2.7 GB) take 373 us to read
// (7.2 TB/s) and 840 to scale into other memory (6.4 TB/s); a tensor and its
// result that start at different places within 16 bytes go value by value
// (13 to 19% slower for 0.6 and 1.2 GB clipped).
//
// Sums: a thread adds the values of a 16-byte vector in fp32, and those sums and
// the tiles' in fp32 with the rounding errors carried (two words); the threads'
// sums are added in fp64 in an order that the sizes, the tensors' starts
// within 16 bytes and the device fix.  A tile's sum below 2^-92 may have lost
// terms to fp32's range (64 squares below 2^-126), one above 2^100 nearly so: it
// is taken again from values times a power of two (618 us where all are).  (fp32
// numbers below 2^-126 count as 0.)
#pragma once

#include "row_kernels.cuh"

namespace gbce {

// 8 vectors a thread and 4 CTAs an SM: 1.3e9 values read in 379 us, clipped in 1257 (4 vectors: 402 and 1279
// with 6 CTAs, 390 and 1318 with 8; 3 CTAs of 8 vectors: 383 and 1270)
constexpr int kNormThreads = 256;
constexpr int kNormCtasPerSm = 4;
constexpr int kNormVecs = 8;                             // 16-byte vectors of a tile that a thread holds
constexpr int64_t kNormTileVecs = kNormThreads * kNormVecs;
constexpr int kNormSmallTable = 64, kNormTable = 1024;   // tensors of a launch
constexpr float kNormLow = 0x1p-92f, kNormHigh = 0x1p100f;
constexpr float kNormUp = 0x1p64f, kNormDown = 0x1p-70f;

enum NormKind { kNormTwo = 0, kNormOne = 1, kNormMax = 2 };

template <int N>
struct NormTable {
    const char *in[N];
    char *out[N];
    int64_t values[N];
    int first[N + 1];      // tiles before each tensor's; first[tensors]: all
    unsigned char type[N];
    int tensors;
};

template <typename T>
struct NormGeom {
    int head;       // values before the first 16-byte boundary
    int64_t vecs, tail_start, values;
};

template <typename T>
__host__ __device__ __forceinline__ NormGeom<T> norm_geom(const void *p, int64_t values)
{
    constexpr int V = 16 / sizeof(T);
    NormGeom<T> g;
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
    g.head = mis ? (16 - mis) / static_cast<int>(sizeof(T)) : 0;
    if (g.head > values)
        g.head = static_cast<int>(values);
    g.vecs = (values - g.head) / V;
    g.tail_start = g.head + g.vecs * V;
    g.values = values;
    return g;
}

// The tensor that a tile is of: the last one whose first tile is not behind it.
template <int N>
__device__ __forceinline__ int norm_tensor(const NormTable<N> &a, int tile)
{
    int lo = 0, hi = a.tensors;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.first[mid] <= tile)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// What a thread has seen: a compensated sum and the sums out of its range, or
// the largest magnitude's bits (a NaN's are above all others).
struct NormSum {
    float sum = 0.f, carry = 0.f;
    double more = 0.0;
    unsigned top = 0;
};

template <int KIND>
__device__ __forceinline__ void norm_value(float x, float &s, unsigned &top)
{
    if constexpr (KIND == kNormTwo)
        s = fmaf(x, x, s);
    else if constexpr (KIND == kNormOne)
        s += fabsf(x);
    else
        top = max(top, __float_as_uint(x) & 0x7fffffffu);
}

// sum += s, its rounding error to carry (exact where both are finite).
__device__ __forceinline__ void norm_carry(float &sum, float &carry, float s)
{
    const float t = sum + s;
    carry += sum >= s ? (sum - t) + s : (s - t) + sum;
    sum = t;
}

// Adds the values of a vector, times `by` if SCALED: in fp32 within it, vector after vector with the errors
// carried.  A chain of a tile's 64 values was 4 to 6e-8 of the sum too low for 16-bit types, whatever their
// number: the last bits of their short squares are not spread evenly and round down more often than up.  Chains
// of 8 leave 0.7e-8 (bf16) and 1.5e-8 (fp16).
template <int KIND, typename T, bool SCALED>
__device__ __forceinline__ void norm_vector(const uint4 &raw, float by, float &s, float &carry, unsigned &top)
{
    using E = Elem<T>;
    constexpr int V = E::kPerVec;
    float f[V], of_vec = 0.f;
    E::unpack(raw, f);
#pragma unroll
    for (int e = 0; e < V; ++e)
        norm_value<KIND>(SCALED ? f[e] * by : f[e], of_vec, top);
    if constexpr (KIND != kNormMax)
        norm_carry(s, carry, of_vec);
}

// Adds one tile's sum, or tells that it is out of range.
template <int KIND>
__device__ __forceinline__ bool norm_add(NormSum &a, float s, float carry)
{
    if constexpr (KIND == kNormMax)
        return true;
    if (!(s < kNormHigh) || (KIND == kNormTwo && s < kNormLow))
        return false;
    norm_carry(a.sum, a.carry, s);
    a.carry += carry;
    return true;
}

template <int KIND, typename T>
__device__ __forceinline__ void norm_tile(const void *p, int64_t values, int64_t tile, NormSum &sum)
{
    using E = Elem<T>;
    const NormGeom<T> g = norm_geom<T>(p, values);
    const T *x = static_cast<const T *>(p);
    const uint4 *v = reinterpret_cast<const uint4 *>(x + g.head);
    const uint4 *mine = v + tile * kNormTileVecs + threadIdx.x;
    const int64_t left = g.vecs - tile * kNormTileVecs - static_cast<int>(threadIdx.x);  // of this thread's on
    const int here = static_cast<int>(left < kNormTileVecs ? left : kNormTileVecs);
    const auto load = [&](int i) {
        return i * kNormThreads < here ? __ldg(mine + i * kNormThreads) : make_uint4(0, 0, 0, 0);
    };
    uint4 raw[kNormVecs];
#pragma unroll
    for (int i = 0; i < kNormVecs; ++i)
        raw[i] = load(i);
    float s = 0.f, carry = 0.f, edge = 0.f;
    if (tile == 0) {  // up to 14 values before and behind the vectors
        const int tail = static_cast<int>(g.values - g.tail_start);
        const int i = static_cast<int>(threadIdx.x);
        if (i < g.head)
            edge = E::load(x + i);
        else if (i - g.head < tail)
            edge = E::load(x + g.tail_start + (i - g.head));
        norm_value<KIND>(edge, s, sum.top);
    }
#pragma unroll
    for (int i = 0; i < kNormVecs; ++i)
        norm_vector<KIND, T, false>(raw[i], 1.f, s, carry, sum.top);
    if (!norm_add<KIND>(sum, s, carry)) {
        unsigned any = __float_as_uint(edge);
#pragma unroll
        for (int i = 0; i < kNormVecs; ++i)
            any |= raw[i].x | raw[i].y | raw[i].z | raw[i].w;
        if (any) {  // not the zeros of rows that no token used
            const float by = s < kNormLow ? kNormUp : kNormDown;
            s = carry = 0.f;
            norm_value<KIND>(edge * by, s, sum.top);
            // read again, one by one: kept, the vectors spilled 416 bytes, and two at a time cost the common path 5 us
            // of 373 (this one 580 us for 618 with 1.3e9 values of 1e-16)
#pragma unroll 1
            for (int i = 0; i < kNormVecs; ++i)
                norm_vector<KIND, T, true>(load(i), by, s, carry, sum.top);
            const double back = 1.0 / static_cast<double>(by);
            const double all = static_cast<double>(s) + static_cast<double>(s < INFINITY ? carry : 0.f);
            sum.more += all * (KIND == kNormTwo ? back * back : back);
        }
    }
}

// Sum (or maximum, a NaN above all) over the CTA, in thread 0.
template <int KIND>
__device__ __forceinline__ double norm_reduce(double v)
{
    __shared__ double part[kNormThreads / 32];
    const auto join = [](double a, double b) {
        return KIND == kNormMax ? (a >= b || a != a ? a : b) : a + b;
    };
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v = join(v, __shfl_xor_sync(0xffffffffu, v, off));
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = part[0];
        for (int w = 1; w < kNormThreads / 32; ++w)
            v = join(v, part[w]);
    }
    return v;
}

// One number a CTA: its tiles' sum or maximum.
template <int KIND, int N>
__global__ void __launch_bounds__(kNormThreads, kNormCtasPerSm) norm_parts_kernel(const __grid_constant__ NormTable<N> a, double *part)
{
    wait_prerequisite_grid();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    NormSum sum;
    const int tiles = a.first[a.tensors];
    for (int tile = blockIdx.x; tile < tiles; tile += static_cast<int>(gridDim.x)) {
        const int i = norm_tensor(a, tile);
        const int64_t at = tile - a.first[i];
        switch (a.type[i]) {
        case 0: norm_tile<KIND, float>(a.in[i], a.values[i], at, sum); break;
        case 1: norm_tile<KIND, __nv_bfloat16>(a.in[i], a.values[i], at, sum); break;
        default: norm_tile<KIND, __half>(a.in[i], a.values[i], at, sum);
        }
    }
    double v = KIND == kNormMax ? static_cast<double>(__uint_as_float(sum.top))
                                : static_cast<double>(sum.sum) + static_cast<double>(sum.carry) + sum.more;
    v = norm_reduce<KIND>(v);
    if (threadIdx.x == 0)
        part[blockIdx.x] = v;
}

// The sum or maximum of the CTAs' numbers, in thread 0.
template <int KIND>
__device__ __forceinline__ double norm_total(const double *part, int parts)
{
    double v = 0.0;
    for (int i = threadIdx.x; i < parts; i += kNormThreads) {
        const double p = __ldcg(part + i);
        v = KIND == kNormMax ? (v >= p || v != v ? v : p) : v + p;
    }
    return norm_reduce<KIND>(v);
}

template <int KIND>
__device__ __forceinline__ double norm_root(double v)
{
    return KIND == kNormTwo ? sqrt(v) : v;
}

template <int KIND>
__global__ void __launch_bounds__(kNormThreads) norm_finish_kernel(const double *part, int parts, float *norm,
                                                                   double *total)
{
    wait_prerequisite_grid();
    const double n = norm_total<KIND>(part, parts);
    if (threadIdx.x == 0) {
        *norm = static_cast<float>(norm_root<KIND>(n));
        if (total)
            *total = n;
    }
}

// f as two fp32 factors, the second a power of two: 1, or 2^-100 where f is
// below fp32's normal numbers.
struct NormFactor {
    float f, power;
    bool copy;
};

template <typename T>
__device__ __forceinline__ T scaled(T x, const NormFactor &by)
{
    if (!by.copy)
        Elem<T>::store(&x, Elem<T>::load(&x) * by.f * by.power);
    return x;
}

// n values of memory that starts at another place within 16 bytes than its
// result: one value at a time, kNormValues of a thread in flight, from a whole
// line of the result on, so that a warp's store fills its sectors.
constexpr int kNormValues = 16;

template <typename T>
__device__ __forceinline__ void scale_apart(const T *x, T *y, int n, const NormFactor &by)
{
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(y) & 127u) / static_cast<int>(sizeof(T));
    const int whole = mis ? 128 / static_cast<int>(sizeof(T)) - mis : 0, lead = whole < n ? whole : n;
    if (static_cast<int>(threadIdx.x) < lead)
        y[threadIdx.x] = scaled(x[threadIdx.x], by);
#pragma unroll 1
    for (int i0 = lead + static_cast<int>(threadIdx.x); i0 < n; i0 += kNormValues * kNormThreads) {
        T raw[kNormValues];
#pragma unroll
        for (int i = 0; i < kNormValues; ++i)
            raw[i] = i0 + i * kNormThreads < n ? x[i0 + i * kNormThreads] : T{};
#pragma unroll
        for (int i = 0; i < kNormValues; ++i)
            if (i0 + i * kNormThreads < n)
                y[i0 + i * kNormThreads] = scaled(raw[i], by);
    }
}

template <typename T>
__device__ __forceinline__ void scale_tile(const void *p, void *q, int64_t values, int64_t tile, const NormFactor &by)
{
    using E = Elem<T>;
    constexpr int V = E::kPerVec;
    const NormGeom<T> g = norm_geom<T>(p, values);
    const T *x = static_cast<const T *>(p);
    T *y = static_cast<T *>(q);
    if (tile == 0) {
        const int tail = static_cast<int>(g.values - g.tail_start);
        const int i = static_cast<int>(threadIdx.x);
        const int64_t at = i < g.head ? i : g.tail_start + (i - g.head);
        if (i < g.head + tail)
            y[at] = scaled(x[at], by);
    }
    if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15u) == 0) {
        const int64_t at = tile * kNormTileVecs + threadIdx.x;
        const uint4 *v = reinterpret_cast<const uint4 *>(x + g.head) + at;
        uint4 *o = reinterpret_cast<uint4 *>(y + g.head) + at;
        const int here = static_cast<int>(g.vecs - at < kNormTileVecs ? g.vecs - at : kNormTileVecs);
        uint4 raw[kNormVecs];
#pragma unroll
        for (int i = 0; i < kNormVecs; ++i)
            raw[i] = i * kNormThreads < here ? __ldcs(v + i * kNormThreads) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kNormVecs; ++i) {
            float w[V];
            E::unpack(raw[i], w);
#pragma unroll
            for (int e = 0; e < V; ++e)
                w[e] = w[e] * by.f * by.power;
            const uint4 r = by.copy ? raw[i] : E::pack(w);
            if (i * kNormThreads < here)
                __stcs(o + i * kNormThreads, r);
        }
        return;
    }
    const int64_t at = g.head + tile * kNormTileVecs * V;
    scale_apart(x + at, y + at, static_cast<int>(g.tail_start - at < kNormTileVecs * V ? g.tail_start - at : kNormTileVecs * V), by);
}

// The tiles in the opposite order: those that the norm read last are still in L2.
template <int KIND, int N>
__global__ void __launch_bounds__(kNormThreads, kNormCtasPerSm) norm_scale_kernel(const __grid_constant__ NormTable<N> a, const double *part,
                                                                  int parts, float *norm, double max_norm, double eps,
                                                                  bool in_place)
{
    wait_prerequisite_grid();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // one thread forms the factor: fp64 is slow here, and nothing of it is left to the loop
    __shared__ NormFactor shared;
    const double n = norm_total<KIND>(part, parts);
    if (threadIdx.x == 0) {
        const double root = norm_root<KIND>(n);
        if (norm && blockIdx.x == 0)
            *norm = static_cast<float>(root);
        double f = max_norm / (root + eps);
        f = f >= 1.0 ? 1.0 : f;  // a NaN stays one
        const bool low = f > 0.0 && f < 0x1p-126;
        shared = {static_cast<float>(low ? f * 0x1p100 : f), low ? 0x1p-100f : 1.f, f == 1.0};
    }
    __syncthreads();
    const NormFactor by = shared;
    if (in_place && by.copy)
        return;
    const int tiles = a.first[a.tensors];
#pragma unroll 1
    for (int tile = tiles - 1 - static_cast<int>(blockIdx.x); tile >= 0; tile -= static_cast<int>(gridDim.x)) {
        const int i = norm_tensor(a, tile);
        const int64_t at = tile - a.first[i];
        switch (a.type[i]) {
        case 0: scale_tile<float>(a.in[i], a.out[i], a.values[i], at, by); break;
        case 1: scale_tile<__nv_bfloat16>(a.in[i], a.out[i], a.values[i], at, by); break;
        default: scale_tile<__half>(a.in[i], a.out[i], a.values[i], at, by);
        }
    }
}

}  // namespace gbce
