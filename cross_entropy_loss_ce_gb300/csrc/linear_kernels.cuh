// The output layer's loss without its logits: hidden states H [n, K] times
// weights W [V, K] in tiles on the tensor cores, each tile's logits consumed
// where they are made (tensor memory) and never written out.
//
//   forward   x = H W^T; per row the online (s, d) pair of the softmax over each
//             256-column tile, merged over the tiles: lse = m + ln d, and the row
//             loss lse - x_y (linear_ce_fwd); or the arg max and its
//             log-probability (linear_greedy).
//   backward  in pieces of the vocabulary: G = (exp(x - lse) - onehot) r from a
//             second product (16-bit, the one rounding between the products),
//             then dW_piece = G^T H, complete, and dH += G W_piece in fp32.
//
// pair_gemm_kernel does every product: pairs of CTAs (cta_group::2) on 256 x 256
// tiles, one CTA holding 128 rows of A, 128 of B's 256 rows, and 128 x 256
// sums.  A producer thread per CTA keeps a ring of 64-wide operand tiles filled
// by TMA, one thread of the pair issues the matrix instructions, and eight warps
// per CTA empty one accumulator while the other one fills (2 x 256 columns, all
// of tensor memory).  The 256 x 256 pair tile reads 64 KB per 2 x 16.8 MFLOP
// k-step, half of what two 128 x 256 tiles would take from L2.
//
// The tensor cores cut each addition short instead of rounding it, toward zero,
// which over a K of 4096 adds up to 40 steps of fp32 in a logit.  Two things
// keep that out of the results.  The logit that a row's answer hangs on (the
// target's, the arg max's) is formed again as an fp32 dot product of two rows
// (0.5% of the time at 8192 rows), and the sums leave its term out, so that the
// loss ln(1 + others / e^x_y) of a likely target and (p_y - 1) keep their
// precision (the backward takes p_y from the row's loss: an fp32 lse of 20 has
// lost a loss of 1e-6).  And logits are summed in tensor memory over kChunk k-steps (1024
// of K) at a time, these sums in registers.  Emptying an accumulator takes
// tensor-memory cycles from the running instructions: 8192 x 128256, K 4096
// takes 4.90 ms unsplit, 5.04-5.22 in runs of 1024, 5.29 of 512, 5.86 of 256.
// The gradient products and their logits end in 16 bits; they are split where the
// axis is so long that what is cut off comes near half a step of that type.  A sum
// of one sign loses 0.6 to 0.8 of a step of 2^-23 for each 16 of the axis (measured:
// a logit of 32 from K = 131072 was low by 0.024, the hidden gradient of 524288
// classes by 2.3e-3 of its sums, the weights' of 262144 rows by 1.6e-3; half a step
// of fp16 is 4.9e-4).  So sums over classes and rows are split after 16384 (fp16) and
// 131072 (bf16) of them, which lose a quarter of half a step at most, and logits
// after 2048 and 16384 of K: those of 32 move their p by less than half a step.
//
// skinny_kernel is the forward for at most 64 rows, where reading W once is the
// whole cost: W's rows take the M side of the instruction, so a tile is 128
// vocabulary rows of any number of hidden states, and each CTA streams every
// gridDim-th tile through a 200 KB ring.  The last, partial round of tiles runs
// at the same bandwidth: the CTAs that have one hold enough loads in flight.
//
// Rows whose target is ignore_index take part in nothing (but where skinny_kernel
// reads the hidden states as they stand): lin_prep_kernel lists the others in order and lin_gather_kernel packs their hidden states (zeros up
// to the next multiple of 256 rows), so the products run over counted rows only.
#pragma once

#include "row_kernels.cuh"
#include "tensor.cuh"

namespace gbce {

constexpr int kPairM = 256, kPairN = 256, kPairK = 64;  // tile of a CTA pair
constexpr int kPairStages = 6;
constexpr int kPairStageBytes = 2 * 128 * kPairK * 2;   // per CTA: 128 rows of A and of B
constexpr int kPairThreads = 384;
constexpr int kPairSmem = kPairStages * kPairStageBytes + 1024;
constexpr int kChunk = 16;                              // k-steps of a logit summed in tensor memory
constexpr int kGradRun = 32, kSumRun = 256;             // ... of the backward's logits and of its sums in fp16;
constexpr int kBf16Runs = 8;                            // in bf16 8 times as many
constexpr int kBand = 8;                                // tiles of M that share a sweep over N

enum class Epi { Stats, Greedy, Grad, Both };  // Both: the two gradient products

struct PairArgs {
    CUtensorMap a, b;
    const int *n_ptr;   // counted rows (device), NULL: n_host
    int n_host;
    int tiles_m;        // dW: tiles of the piece's classes; else from n
    int tiles_n;
    int kblocks;        // 64-wide steps along K; dW: from n
    int run;            // RUNS: k-steps summed in tensor memory at a time
    float *runs;        // ... sums of earlier runs, kPairM x kPairN for each pair
    int b_row0;         // Grad, dH: the piece's first row of W
    unsigned *fail;
    int drop_copy;      // failure-path tests: the k-step whose A block CTA 0 leaves out, else -1
    // Stats, Greedy
    float2 *part;       // Stats: [row][ldp] (s, d) pairs, one for each 128 columns
    float4 *best;       // Greedy: [row][ldp] (maximum, others' sum, arg max)
    int64_t ldp;
    const int *tgt;
    int64_t V;          // columns of this launch's logits (vocabulary, or end of it) from row 0 of W
    // Grad
    const float *l2, *rs, *gy;  // lse log2e, factor and target's entry of each row
    void *g;
    int64_t ldg;
    // dH and dW
    const float *alpha;
    void *out;
    int64_t ldo;
    int64_t rows, cols; // valid rows (dW) and columns of out
    int vec;            // out allows 16-byte stores
    const int *idx;     // dH: the row of out that a packed row belongs to
    float *acc;         // dH: fp32 sums over pieces
    int first, last;    // dH: the first piece does not read acc, the last one writes out
    float *slices;      // kSplitUnits sums of kPairM x kPairN, for split tiles
    unsigned *arrived;  // ... and 16 counters a split tile, zero before and after
};

// The tiles of a product that fill no whole wave of the CTA pairs, cut along K:
// 248 tiles on 76 pairs take 4 waves, of which the last is a quarter full; its
// 20 tiles in 3 slices each make it a third of a wave.  The first `whole` tiles
// are done as they are; then come `tail` tiles in `slices` slices, slice by
// slice, whose sums go to memory; whichever warp is the last to write its 32 x 128
// part of a tile adds the slices of that part, in order, and finishes it.
struct Split {
    int whole, tail, slices;
};

constexpr int kSplitUnits = 4 * 80;  // slices of a launch, at most
constexpr int kSplitMax = 8;         // slices of a tile, at most
constexpr int kSplitCounters = 2 * (kSplitUnits / 2) * 16;  // 16 for each split tile of dH and of dW

// Costs in k-steps of one tile: a slice takes its steps and about 6 more to be
// written, and 8 to be read again (3 cut too finely: 1500 x 3000, K 2048 took 78 us
// backward, 66 with 8).  The tail is the last, partial wave, or that and
// a whole one.  A warp weighs up all choices at once, one in each lane.
__device__ __forceinline__ Split split_of(int tiles, int pairs, int kblocks)
{
    const int lane = threadIdx.x & 31;
    const int s = 2 + (lane & 7), rest = tiles % pairs, tail = rest + (lane & 8 ? pairs : 0);
    int64_t cost = static_cast<int64_t>((tiles + pairs - 1) / pairs) * kblocks;  // no slices
    if (lane < 16) {
        const bool fits = rest && tail <= tiles && s <= kSplitMax && 4 * s <= kblocks && tail * s <= kSplitUnits;
        const int64_t sliced = static_cast<int64_t>((tiles - tail) / pairs) * kblocks +
                               static_cast<int64_t>((tail * s + pairs - 1) / pairs) * ((kblocks + s - 1) / s + 6) + 8 * s;
        cost = fits ? sliced : INT64_MAX;
    }
    int best = lane;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const int64_t c = __shfl_xor_sync(0xffffffffu, cost, off);
        const int b = __shfl_xor_sync(0xffffffffu, best, off);
        if (c < cost || (c == cost && b > best)) {  // of equal ones the last: lanes 16 .. 31 cut nothing
            cost = c;
            best = b;
        }
    }
    if (best >= 16)
        return Split{tiles, 0, 1};
    const int slices = 2 + (best & 7), cut = rest + (best & 8 ? pairs : 0);
    return Split{tiles - cut, cut, slices};
}

// One CTA pair's share of a tile: k-steps k0 .. k1, and where a slice's sums go (-1: a whole tile).
struct Unit {
    int tile, k0, k1, slice;
};

__device__ __forceinline__ Unit unit_at(int u, const Split &sp, int kblocks)
{
    if (u < sp.whole)
        return Unit{u, 0, kblocks, -1};
    const int v = u - sp.whole, s = v / sp.tail, t = v - s * sp.tail;
    return Unit{sp.whole + t, static_cast<int>(int64_t{kblocks} * s / sp.slices),
                static_cast<int>(int64_t{kblocks} * (s + 1) / sp.slices), t * sp.slices + s};
}

// Lets the next kernel of the stream be set up while this one runs.  Every
// kernel of a call then waits for its predecessor before it reads or ends, so
// that a kernel's end means the end of all before it.
__device__ __forceinline__ void next_kernel_may_start()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int &m, int &n)
{
    const int band = t / (kBand * tiles_n);
    const int r = t - band * kBand * tiles_n;
    const int rows = min(kBand, tiles_m - band * kBand);
    n = r / rows;
    m = band * kBand + (r - n * rows);
}

// exp2 shift of a maximum, finite for an empty part.
__device__ __forceinline__ float finite_shift(float m) { return m == -INFINITY ? 0.f : shift_of(m); }

// A sum about the maximum `from`, about the larger maximum `to`.  An empty part
// (-inf) holds 0, or a NaN that has to stay.
__device__ __forceinline__ float rescaled(float d, float from, float to)
{
    return from == -INFINITY ? d : d * exp2f(shift_of(from) - shift_of(to));
}

// exp2 of a maximum about its own shift: 1 up to the shift's rounding.
__device__ __forceinline__ float self_term(float m) { return exp2_shift(m, shift_of(m)); }

// The arg max keeps its sum without the maximum's own term: the log-probability
// -ln(1 + d / self_term(m)) of a nearly certain token keeps its precision.  The
// sum about a new maximum `to`, which the old one's term now joins:
__device__ __forceinline__ float rescaled_others(float d, float from, float to)
{
    return from == -INFINITY ? d : (d + self_term(from)) * exp2f(shift_of(from) - shift_of(to));
}

// Merge of two (maximum, others, index) triples: the lower index of equal maxima.
__device__ __forceinline__ void best_merge(float &m, float &d, int &i, float m2, float d2, int i2)
{
    if (m2 > m || (m2 == m && i2 < i)) {
        d = d2 + rescaled_others(d, m, m2);
        m = m2;
        i = i2;
    } else {
        d += rescaled_others(d2, m2, m);
    }
}

// A sum about the shift `from`, about the larger shift `to` (-inf: empty, or a
// NaN that has to stay).
__device__ __forceinline__ float shifted(float d, float from, float to)
{
    return from == -INFINITY ? d : d * exp2f(from - to);
}

// 32 logits of one row, x[OFF ..], columns c0 .. c0 + 31 of W's rows, into the
// running maximum m and sum d = sum exp2(x log2e - fl(m log2e)) (GREEDY: of all
// but the maximum, whose column is `best`).
template <bool GREEDY, int OFF, int N>
__device__ __forceinline__ void stats_chunk(float (&x)[N], int c0, int limit, float &m, float &d, int &best)
{
    if (c0 + 32 > limit) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            x[OFF + i] = c0 + i < limit ? x[OFF + i] : -INFINITY;
    }
    // four chains each for the maximum and the sum: two warps a scheduler do not
    // hide the latency of one (8192 x 32000, K 512, where this work outlasts the
    // tile's products: forward 199 us with one and two chains, 184 so)
    float top[4] = {x[OFF], x[OFF + 1], x[OFF + 2], x[OFF + 3]};
#pragma unroll
    for (int i = 4; i < 32; ++i)
        top[i & 3] = fmaxf(top[i & 3], x[OFF + i]);
    const float mc = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    if (mc > m) {
        if constexpr (GREEDY) {
            int at = 31;
#pragma unroll
            for (int i = 31; i >= 0; --i)
                at = x[OFF + i] == mc ? i : at;
            best = c0 + at;
            d = rescaled_others(d, m, mc);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                x[OFF + i] = i == at ? -INFINITY : x[OFF + i];
        } else {
            d = rescaled(d, m, mc);
        }
        m = mc;
    }
    const float s = finite_shift(m);
    float sum[4] = {};
#pragma unroll
    for (int i = 0; i < 32; ++i)
        sum[i & 3] += exp2_shift(x[OFF + i], s);
    d += (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// A warp's 32 x 32 block of finished values, a thread one row, rounded once and
// written to rows of `out` (row_of(r): where row r of the block goes, for r <
// rows; columns col .. below cols).  A thread's own row would make each store of
// a warp touch 32 lines (the weights' gradient of one row of 128256 x 2048, which
// is all stores: 250 us, 171 so); turned around in `turn`, the warp's own, 4 lanes
// write 64 bytes of a row, or 32 lanes one row where it allows no 16-byte stores.
constexpr int kTurnStride = 40;  // 80 bytes: 16-byte accesses of 8 rows meet in no bank

template <typename T>
__device__ __forceinline__ void turn_block(const float (&f)[32], T *turn)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float *p = f + 8 * q;
        *reinterpret_cast<uint4 *>(turn + lane * kTurnStride + 8 * q) =
            make_uint4(Elem<T>::pack2(p[0], p[1]), Elem<T>::pack2(p[2], p[3]),
                       Elem<T>::pack2(p[4], p[5]), Elem<T>::pack2(p[6], p[7]));
    }
    __syncwarp();
}

// A whole block to rows that allow 16-byte stores: `to[i]` is where this lane's
// 8 columns of row 8 i + lane / 4 go.  Without bounds checks and addresses formed
// anew for each block the weights' gradient of one row of 128256 x 2048 takes
// 137 us instead of 171 (its 525 MB are 78 us at the copy bandwidth; what is left
// is the latency from one accumulator to the next).
template <typename T>
__device__ __forceinline__ void store_whole_block(T *const (&to)[4], int offset, const float (&f)[32], T *turn)
{
    const int lane = threadIdx.x & 31;
    turn_block(f, turn);
    const T *from = turn + (lane >> 2) * kTurnStride + 8 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(to[i] + offset) = *reinterpret_cast<const uint4 *>(from + 8 * i * kTurnStride);
}

template <typename T, typename RowOf>
__device__ __forceinline__ void store_block(T *out, int64_t ldo, int64_t col, int64_t cols, int rows,
                                            const float (&f)[32], bool vec, T *turn, RowOf row_of)
{
    const int lane = threadIdx.x & 31;
    turn_block(f, turn);
    if (vec) {
        const int64_t c = col + 8 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2);
            if (r >= rows || c >= cols)
                continue;
            const T *from = turn + r * kTurnStride + 8 * (lane & 3);
            T *to = out + row_of(r) * ldo + c;
            if (c + 8 <= cols) {
                *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
            } else {
                for (int e = 0; c + e < cols; ++e)
                    to[e] = from[e];
            }
        }
    } else if (col + lane < cols) {
#pragma unroll 8
        for (int r = 0; r < 32; ++r)
            if (r < rows)
                out[row_of(r) * ldo + col + lane] = turn[r * kTurnStride + lane];
    }
}

// Sums that a kernel keeps for itself lie as the threads hold them: 16 parts of a
// tile (a warp of a CTA each), 4 blocks of 32 x 32 a part, 16 bytes of each of
// the 32 lanes together.
__device__ __forceinline__ float4 *block_at(float *base, int64_t tile, int part, int c)
{
    return reinterpret_cast<float4 *>(base + ((tile * 16 + part) * 4 + c) * 1024) + (threadIdx.x & 31);
}

__device__ __forceinline__ void add_block(float (&f)[32], const float4 *from)
{
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const float4 v = __ldcg(from + 32 * q);
        f[4 * q] += v.x;
        f[4 * q + 1] += v.y;
        f[4 * q + 2] += v.z;
        f[4 * q + 3] += v.w;
    }
}

__device__ __forceinline__ void put_block(float4 *to, const float (&f)[32])
{
#pragma unroll
    for (int q = 0; q < 8; ++q)
        to[32 * q] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
}

// A block of a gradient product whose sums over K are complete: dW times alpha to
// its rows; dH added to what earlier pieces left and kept for the next one, or
// times alpha to the rows they belong to.
template <bool WEIGHT, typename T>
__device__ __forceinline__ void finish_block(const PairArgs &a, float (&f)[32], int tile, int part, int c,
                                             int64_t row0, int64_t col, int64_t rows, float alpha, T *turn)
{
    if (col >= a.cols || row0 >= rows)
        return;
    if constexpr (!WEIGHT) {
        if (!a.first)
            add_block(f, block_at(a.acc, tile, part, c));
        if (!a.last) {
            put_block(block_at(a.acc, tile, part, c), f);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
        f[i] *= alpha;
    store_block(static_cast<T *>(a.out), a.ldo, col, a.cols, static_cast<int>(min(rows - row0, int64_t{32})), f, a.vec,
                turn, [&](int r) { return WEIGHT ? row0 + r : int64_t{a.idx[row0 + r]}; });
}

// RUNS: axes longer than a.run (the others' tiles are one run each; the loop over runs
// in their kernel too cost 2% of the backward of 1 row of 128256 x 2048 and of 256 of 32000)
template <Epi E, bool RUNS, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_gemm_kernel(const __grid_constant__ PairArgs a, const __grid_constant__ PairArgs w)
{
    // Both: `a` is dH = G W (G K-major, W MN-major), then `w` is dW = G^T H (both
    // MN-major); either may have no tiles.  Else `a` alone, both operands K-major.
    constexpr bool BOTH = E == Epi::Both;
    constexpr bool CHUNKED = E == Epi::Stats || E == Epi::Greedy;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kIdesc = mma_idesc(kBf16, false, BOTH, kPairM, kPairN);
    constexpr uint32_t kIdescW = mma_idesc(kBf16, true, true, kPairM, kPairN);

    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kPairStages + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ int dead_word;
    __shared__ __align__(16) T turn[CHUNKED ? 1 : 8][CHUNKED ? 1 : 32 * kTurnStride];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    volatile int *dead = &dead_word;
    const uint32_t ring = (smem_addr(dyn) + 1023u) & ~1023u;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kPairStages;
    const uint32_t tfull = empty + 8 * kPairStages, tempty = tfull + 16;

    if (threadIdx.x == 0) {
        dead_word = 0;
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(full + 8 * i, 1);   // the leader's expect_tx; both CTAs' bytes count on it
            mbar_init(empty + 8 * i, 1);  // the commit of the instructions that read the slot
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, 16);  // eight warps of each CTA
        }
        fence_barrier_init();
        prefetch_map(&a.a);
        prefetch_map(&a.b);
        if (BOTH) {
            prefetch_map(&w.a);
            prefetch_map(&w.b);
        }
    }
    if (warp == 2)
        tmem_alloc<2>(smem_addr(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    next_kernel_may_start();
    wait_prerequisite_grid();

    const int n = a.n_ptr ? *a.n_ptr : a.n_host;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int tiles_m = (n + kPairM - 1) / kPairM;
    const int steps_w = (n + kPairK - 1) / kPairK;  // dW's k-steps run over the rows
    const Split sp = BOTH ? split_of(tiles_m * a.tiles_n, pairs, a.kblocks) : Split{tiles_m * a.tiles_n, 0, 1};
    const Split spw = BOTH ? split_of(w.tiles_m * w.tiles_n, pairs, steps_w) : Split{0, 0, 1};
    const int units = sp.whole + sp.tail * sp.slices, units_w = spw.whole + spw.tail * spw.slices;
    // body(part of a tile, its row and column of tiles, is it dW's) until it is false;
    // dW's parts go first to the pairs that the last round of dH's left out
    const auto each_unit = [&](auto &&body) {
        int tm, tn;
        for (int u = pair; u < units; u += pairs) {
            const Unit un = unit_at(u, sp, a.kblocks);
            tile_at(un.tile, tiles_m, a.tiles_n, tm, tn);
            if (!body(un, tm, tn, false))
                return;
        }
        for (int u = (pair + pairs - units % pairs) % pairs; BOTH && u < units_w; u += pairs) {
            const Unit un = unit_at(u, spw, steps_w);
            tile_at(un.tile, w.tiles_m, w.tiles_n, tm, tn);
            if (!body(un, tm, tn, true))
                return;
        }
    };

    // 128 sums a thread want more than the launch's 168 registers: the first
    // four warps give some of theirs up (64 x 128 + 216 x 256 <= 168 x 384)
    if (warp < 4) {
        if constexpr (CHUNKED)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 0 && lane == 0) {
            // producer: this CTA's halves of A and B
            const uint32_t full0 = map_to_rank(full, 0);
            int slot = 0, steps = 0;
            uint32_t phase = 0;
            each_unit([&](const Unit &un, int tm, int tn, bool dw) {
                const PairArgs &p = BOTH && dw ? w : a;
                const int am = tm * kPairM + static_cast<int>(rank) * 128;
                const int bn = tn * kPairN + static_cast<int>(rank) * 128;
                for (int kb = un.k0; kb < un.k1; ++kb) {
                    if (!bar_wait<true>(empty + 8 * slot, phase ^ 1, dead))
                        return false;
                    if (rank == 0)
                        mbar_arrive_expect_tx(full + 8 * slot, 2 * kPairStageBytes);
                    const uint32_t sa = ring + slot * kPairStageBytes, sb = sa + kPairStageBytes / 2;
                    const uint32_t bar = full0 + 8 * slot;
                    const int k0 = kb * kPairK;
                    if (blockIdx.x == 0 && steps++ == a.drop_copy) {
                        // nothing arrives for A: the waits for this slot run out
                    } else if (BOTH && dw) {
                        tma_load_pair(sa, &p.a, am, k0, bar);
                        tma_load_pair(sa + 8192, &p.a, am + 64, k0, bar);
                    } else {
                        tma_load_pair(sa, &p.a, k0, am, bar);
                    }
                    if constexpr (BOTH) {
                        tma_load_pair(sb, &p.b, bn, p.b_row0 + k0, bar);
                        tma_load_pair(sb + 8192, &p.b, bn + 64, p.b_row0 + k0, bar);
                    } else {
                        tma_load_pair(sb, &p.b, k0, p.b_row0 + bn, bar);
                    }
                    if (++slot == kPairStages) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                return true;
            });
        } else if (warp == 1 && lane == 0 && rank == 0) {
            // the pair's matrix instructions
            int slot = 0, it = 0;
            uint32_t phase = 0;
            each_unit([&](const Unit &un, int, int, bool dw) {
                const uint32_t idesc = BOTH && dw ? kIdescW : kIdesc;
                const uint32_t lbo_a = BOTH && dw ? 8192 : 16, step_a = BOTH && dw ? 128 : 2;
                const int run = CHUNKED ? kChunk : RUNS ? a.run : max(un.k1 - un.k0, 1);  // k-steps that stay in tensor memory
                for (int kb0 = un.k0; kb0 < un.k1 || kb0 == 0; kb0 += run, ++it) {
                    const int acc = it & 1;
                    if (!bar_wait<true>(tempty + 8 * acc, ((it >> 1) & 1) ^ 1, dead))
                        return false;
                    tc_fence_after();
                    const int kb1 = min(kb0 + run, un.k1);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!bar_wait<true>(full + 8 * slot, phase, dead))
                            return false;
                        tc_fence_after();
                        const uint32_t sa = ring + slot * kPairStageBytes, sb = sa + kPairStageBytes / 2;
                        const uint64_t da = smem_desc(sa, lbo_a, 1024);
                        const uint64_t db = smem_desc(sb, BOTH ? 8192 : 16, 1024);
#pragma unroll
                        for (int k = 0; k < kPairK / 16; ++k)  // 16 of K: 32 bytes, or 16 rows of 128 bytes
                            mma_f16<2>(tmem + acc * kPairN, da + k * step_a, db + k * (BOTH ? 128 : 2), idesc,
                                       kb != kb0 || k != 0);
                        mma_commit_pair(empty + 8 * slot);
                        if (++slot == kPairStages) {
                            slot = 0;
                            phase ^= 1;
                        }
                    }
                    mma_commit_pair(tfull + 8 * acc);
                }
                return true;
            });
        }
    } else {
        if constexpr (CHUNKED)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // epilogue: thread = one row of this CTA's 128, 128 of the 256 columns
        const int ew = warp & 3, half = (warp - 4) >> 2;
        const uint32_t tempty0 = map_to_rank(tempty, 0);
        const int limit = static_cast<int>(min(a.V, static_cast<int64_t>(INT32_MAX)));
        [[maybe_unused]] const float alpha = BOTH ? *a.alpha : 1.f;
        int it = 0;
        each_unit([&](const Unit &un, int tm, int tn, bool dw) {
            const PairArgs &p = BOTH && dw ? w : a;
            const int row = tm * kPairM + static_cast<int>(rank) * 128 + ew * 32 + lane;
            const int c0 = tn * kPairN + half * 128;
            const bool live = row < n;
            const uint32_t lanes = tmem + half * 128 + (static_cast<uint32_t>(ew * 32) << 16);
            if constexpr (CHUNKED) {
                float x[128];
                // what a row needs is loaded while its sums are still on their way
                [[maybe_unused]] int y = -1;
                if constexpr (E == Epi::Stats)
                    y = live ? a.tgt[row] - c0 : -1;
                const auto drain = [&](auto first) {
                    const int acc = it & 1;
                    if (!bar_wait<true>(tfull + 8 * acc, (it >> 1) & 1, dead))
                        return false;
                    ++it;
                    tc_fence_after();
                    const uint32_t src = lanes + acc * kPairN;
                    if constexpr (decltype(first)::value) {
                        tmem_ld32_into<0>(src, x);
                        tmem_ld32_into<32>(src + 32, x);
                        tmem_ld32_into<64>(src + 64, x);
                        tmem_ld32_into<96>(src + 96, x);
                        tmem_wait_into(x);
                    } else {
                        uint32_t buf[2][16];
                        tmem_ld16(src, buf[0]);
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            tmem_wait_ld(buf[c & 1]);
                            if (c + 1 < 8)
                                tmem_ld16(src + 16 * (c + 1), buf[(c + 1) & 1]);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                x[16 * c + i] += __uint_as_float(buf[c & 1][i]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive_cluster(tempty0 + 8 * acc);
                    return true;
                };
                if (!drain(std::true_type{}))
                    return false;
                for (int kb0 = kChunk; kb0 < un.k1; kb0 += kChunk)
                    if (!drain(std::false_type{}))
                        return false;
                if constexpr (E == Epi::Stats) {  // the target's term is left out
                    if (y >= 0 && y < 128) {
#pragma unroll
                        for (int i = 0; i < 128; ++i)
                            x[i] = y == i ? -INFINITY : x[i];
                    }
                }
                float m = -INFINITY, d = 0.f;
                int best = 0;
                stats_chunk<E == Epi::Greedy, 0>(x, c0, limit, m, d, best);
                stats_chunk<E == Epi::Greedy, 32>(x, c0 + 32, limit, m, d, best);
                stats_chunk<E == Epi::Greedy, 64>(x, c0 + 64, limit, m, d, best);
                stats_chunk<E == Epi::Greedy, 96>(x, c0 + 96, limit, m, d, best);
                if (live) {
                    const int64_t at = row * a.ldp + 2 * tn + half;
                    if constexpr (E == Epi::Greedy)
                        a.best[at] = make_float4(m, d, __int_as_float(best), 0.f);
                    else
                        a.part[at] = make_float2(m == -INFINITY ? m : shift_of(m), d);
                }
            } else {
                [[maybe_unused]] int y = -1, inside = 0;  // columns with a gradient: none of an unlisted row
                [[maybe_unused]] float l2 = 0.f, rs = 0.f, gy = 0.f;
                if constexpr (E == Epi::Grad)
                    if (live) {
                        y = a.tgt[row] - a.b_row0;
                        inside = limit;
                        l2 = a.l2[row];
                        rs = a.rs[row];
                        gy = a.gy[row];
                    }
                [[maybe_unused]] const int part = static_cast<int>(rank) * 8 + warp - 4;
                // all runs but the last one are added up where this thread alone reads them
                [[maybe_unused]] bool more = false;
                for (int k1 = un.k0 + a.run; RUNS && k1 < un.k1; k1 += a.run) {
                    const int acc = it & 1;
                    if (!bar_wait<true>(tfull + 8 * acc, (it >> 1) & 1, dead))
                        return false;
                    ++it;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        tmem_ld32(lanes + acc * kPairN + 32 * c, r);
                        tmem_wait_ld(r);
                        float f[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            f[i] = __uint_as_float(r[i]);
                        if (more)
                            add_block(f, block_at(a.runs, pair, part, c));
                        put_block(block_at(a.runs, pair, part, c), f);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive_cluster(tempty0 + 8 * acc);
                    more = true;
                }
                const int acc = it & 1;
                if (!bar_wait<true>(tfull + 8 * acc, (it >> 1) & 1, dead))
                    return false;
                ++it;
                tc_fence_after();
                // where this lane's share of each block goes, for blocks that are whole
                const int row0 = row - lane;
                T *to[4];
                bool whole = true;
                if constexpr (BOTH)
                    whole = un.slice < 0 && un.k1 && p.vec && (dw || p.last) && row0 + 32 <= (dw ? p.rows : n) &&
                            c0 + 128 <= p.cols;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    int64_t r = row0 + 8 * i + (lane >> 2);
                    if constexpr (BOTH)
                        if (!dw && whole)
                            r = p.idx[r];
                    to[i] = static_cast<T *>(BOTH ? p.out : a.g) + r * (BOTH ? p.ldo : a.ldg) + c0 + 8 * (lane & 3);
                }
                // one body for all four blocks: unrolled, its code leaves the instruction cache
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t r[32];
                    tmem_ld32(lanes + acc * kPairN + 32 * c, r);
                    tmem_wait_ld(r);
                    const int col = c0 + 32 * c;
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        f[i] = __uint_as_float(r[i]);
                    if (RUNS && more)
                        add_block(f, block_at(a.runs, pair, part, c));
                    if constexpr (E == Epi::Grad) {
                        if (col + 32 <= inside) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                f[i] = exp2_shift(f[i], l2) * rs;
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                f[i] = col + i < inside ? exp2_shift(f[i], l2) * rs : 0.f;
                        }
                        if (y >= col && y < col + 32) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                f[i] = y == col + i ? gy : f[i];
                        }
                        store_whole_block(to, 32 * c, f, turn[warp - 4]);
                    } else if (whole) {
                        if (!dw && !p.first)
                            add_block(f, block_at(p.acc, un.tile, part, c));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            f[i] *= alpha;
                        store_whole_block(to, 32 * c, f, turn[warp - 4]);
                    } else {
                        if (!un.k1) {  // no step: nothing was added up
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                f[i] = 0.f;
                        }
                        if (un.slice >= 0)
                            put_block(block_at(p.slices, un.slice, part, c), f);
                        else if (dw)
                            finish_block<true, T>(p, f, un.tile, part, c, row0, col, p.rows, alpha, turn[warp - 4]);
                        else
                            finish_block<false, T>(p, f, un.tile, part, c, row0, col, n, alpha, turn[warp - 4]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive_cluster(tempty0 + 8 * acc);
                if constexpr (BOTH)
                    if (un.slice >= 0) {
                        // the last of this part's slices to arrive adds them all up
                        const Split &split = dw ? spw : sp;
                        const int t = un.tile - split.whole;
                        unsigned *count = p.arrived + t * 16 + part;
                        unsigned before = 0;
                        __threadfence();
                        __syncwarp();
                        if (lane == 0)
                            before = atomicAdd(count, 1u);
                        before = __shfl_sync(0xffffffffu, before, 0);
                        if (before == static_cast<unsigned>(split.slices - 1)) {
                            __threadfence();
                            if (lane == 0)
                                *count = 0u;  // for the next launch
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                float f[32] = {};
#pragma unroll 2
                                for (int k = 0; k < split.slices; ++k)
                                    add_block(f, block_at(p.slices, t * split.slices + k, part, c));
                                if (dw)
                                    finish_block<true, T>(p, f, un.tile, part, c, row0, c0 + 32 * c, p.rows,
                                                          alpha, turn[warp - 4]);
                                else
                                    finish_block<false, T>(p, f, un.tile, part, c, row0, c0 + 32 * c, n, alpha,
                                                           turn[warp - 4]);
                            }
                        }
                    }
            }
            return true;
        });
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*dead) {
        if (threadIdx.x == 0)
            raise_timeout(a.fail);
        settle_after_failure();
    }
    cluster_arrive();
    cluster_wait();
    if (warp == 2)
        tmem_free<2>(tmem, 512);
}

// ---------------------------------------------------------------------------
// at most 64 rows: W streamed once, its rows on the M side

constexpr int kSkinnyStageW = 128 * 64 * 2;

template <int NG>
__host__ __device__ constexpr int skinny_stage_bytes() { return kSkinnyStageW + NG * 32 * 128; }
template <int NG>
__host__ __device__ constexpr int skinny_stages() { return NG == 1 ? 10 : 8; }
template <int NG>
__host__ __device__ constexpr int skinny_smem() { return skinny_stages<NG>() * skinny_stage_bytes<NG>() + 1024; }
template <int NG>
__host__ __device__ constexpr int skinny_threads() { return 128 + NG * 128; }

struct SkinnyArgs {
    CUtensorMap w;      // W in boxes of 128 rows
    CUtensorMap h;      // hidden states in boxes of 32 NG rows
    const int *n_ptr;
    int n_host;
    int kblocks;
    int64_t V;
    const int *tgt;     // targets of the listed rows, or
    const int64_t *targets;  // ... of all rows as they stand (then CTA 0 clears *fail)
    float2 *part;       // [row][ldp], one for each CTA
    float4 *best;
    int64_t ldp;
    unsigned *fail;
    int drop_copy;      // as in PairArgs, of W
    uint32_t bf16;
};

template <int NG, bool GREEDY>
__global__ void __launch_bounds__(skinny_threads<NG>(), 1) skinny_kernel(const __grid_constant__ SkinnyArgs a)
{
    constexpr int kStages = skinny_stages<NG>();
    constexpr int kStage = skinny_stage_bytes<NG>();
    constexpr int kN = 32 * NG;
    constexpr uint32_t kCols = 2 * kN;

    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ int dead_word;
    __shared__ int tgt[kN];
    __shared__ float sm[NG * 4][32], sd[NG * 4][32];
    __shared__ int si[NG * 4][32];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *dead = &dead_word;
    const uint32_t ring = (smem_addr(dyn) + 1023u) & ~1023u;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kStages;
    const uint32_t tfull = empty + 8 * kStages, tempty = tfull + 16;
    const uint32_t idesc = a.bf16 ? mma_idesc(true, false, false, 128, kN) : mma_idesc(false, false, false, 128, kN);

    if (threadIdx.x == 0) {
        dead_word = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, 4 * NG);
        }
        fence_barrier_init();
        prefetch_map(&a.w);
        prefetch_map(&a.h);
    }
    if (warp == 2)
        tmem_alloc<1>(smem_addr(&tmem_slot), kCols);
    next_kernel_may_start();
    wait_prerequisite_grid();
    const int n = a.n_ptr ? *a.n_ptr : a.n_host;
    if (!GREEDY && threadIdx.x < kN) {
        int64_t y = -1;
        if (static_cast<int>(threadIdx.x) < n)
            y = a.targets ? a.targets[threadIdx.x] : a.tgt[threadIdx.x];
        tgt[threadIdx.x] = y >= 0 && y < a.V ? static_cast<int>(y) : -1;
        if (a.targets && blockIdx.x == 0 && threadIdx.x == 0)
            *a.fail = 0u;  // no wait has given up yet: each takes 2 s to
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    const int all = n > 0 ? static_cast<int>((a.V + 127) / 128) : 0;
    const int first = blockIdx.x, step = gridDim.x;

    if (warp == 0 && lane == 0) {
        const uint64_t once = policy_evict_first(), again = policy_evict_last();
        int slot = 0, steps = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = first; t < all && ok; t += step) {
            for (int kb = 0; kb < a.kblocks; ++kb) {
                if (!(ok = bar_wait<false>(empty + 8 * slot, phase ^ 1, dead)))
                    break;
                const uint32_t sw = ring + slot * kStage, sh = sw + kSkinnyStageW;
                const uint32_t bar = full + 8 * slot;
                mbar_arrive_expect_tx(bar, kStage);
                if (blockIdx.x != 0 || steps++ != a.drop_copy)
                    tma_load(sw, &a.w, kb * 64, t * 128, bar, once);
                tma_load(sh, &a.h, kb * 64, 0, bar, again);
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp == 1 && lane == 0) {
        int slot = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = first; t < all && ok; t += step) {
            for (int kb0 = 0; ok && kb0 < a.kblocks; kb0 += kChunk, ++it) {
                const int acc = it & 1;
                if (!(ok = bar_wait<false>(tempty + 8 * acc, ((it >> 1) & 1) ^ 1, dead)))
                    break;
                tc_fence_after();
                const int kb1 = min(kb0 + kChunk, a.kblocks);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!(ok = bar_wait<false>(full + 8 * slot, phase, dead)))
                        break;
                    tc_fence_after();
                    const uint32_t sw = ring + slot * kStage;
                    const uint64_t da = smem_desc(sw, 16, 1024), db = smem_desc(sw + kSkinnyStageW, 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16<1>(tmem + acc * kN, da + 2 * k, db + 2 * k, idesc, kb != kb0 || k != 0);
                    mma_commit(empty + 8 * slot);
                    if (++slot == kStages) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (ok)
                    mma_commit(tfull + 8 * acc);
            }
        }
    } else if (warp >= 4) {
        // lane = a vocabulary row, column = a hidden state; each thread keeps the
        // running (m, d, index) of its vocabulary rows for 32 hidden states
        const int ew = warp & 3, group = (warp - 4) >> 2;
        float m[32], d[32];
        int best[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            m[j] = -INFINITY;
            d[j] = 0.f;
            best[j] = INT32_MAX;
        }
        const int per = (n + NG - 1) / NG, col0 = group * per;  // of a group's warps
        const int live = min(max(n - col0, 0), per);
        int it = 0;
        bool ok = true;
        for (int t = first; t < all && ok; t += step) {
            float sum[32];
            for (int kb0 = 0; kb0 < a.kblocks; kb0 += kChunk, ++it) {
                const int acc = it & 1;
                if (!(ok = bar_wait<false>(tfull + 8 * acc, (it >> 1) & 1, dead)))
                    break;
                tc_fence_after();
                const uint32_t src = tmem + acc * kN + col0 + (static_cast<uint32_t>(ew * 32) << 16);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t r[16];
                    tmem_ld16(src + 16 * c, r);
                    tmem_wait_ld(r);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        sum[16 * c + j] = kb0 ? sum[16 * c + j] + __uint_as_float(r[j]) : __uint_as_float(r[j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(tempty + 8 * acc);
            }
            if (!ok)
                break;
            const int64_t v = 128 * int64_t{t} + ew * 32 + lane;
            if (v < a.V) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (j < live) {
                        const float x = sum[j];
                        if constexpr (GREEDY) {
                            if (x > m[j]) {
                                d[j] = rescaled_others(d[j], m[j], x);
                                m[j] = x;
                                best[j] = static_cast<int>(v);
                            } else {
                                d[j] += exp2_shift(x, finite_shift(m[j]));
                            }
                        } else {
                            if (tgt[col0 + j] == v)
                                continue;  // the target's term is left out
                            if (x > m[j]) {
                                d[j] = rescaled(d[j], m[j], x);
                                m[j] = x;
                            }
                            d[j] += exp2_shift(x, finite_shift(m[j]));
                        }
                    }
                }
            }
        }
        // each warp turns its 32 x 32 states around in the ring, which is idle once
        // the last accumulator is full: lane j merges the 32 lanes' states of hidden
        // state j
        if (ok && first < all) {
            float *tm = reinterpret_cast<float *>(dyn + (ring - smem_addr(dyn))) + (warp - 4) * 3 * 32 * 33;
            float *td = tm + 32 * 33;
            int *ti = reinterpret_cast<int *>(td + 32 * 33);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                tm[lane * 33 + j] = m[j];
                td[lane * 33 + j] = d[j];
                if (GREEDY)
                    ti[lane * 33 + j] = best[j];
            }
            __syncwarp();
            float mt = tm[lane], dt = 0.f;
            int it = GREEDY ? ti[lane] : 0;
#pragma unroll 8
            for (int l = 1; l < 32; ++l) {
                const float m2 = tm[l * 33 + lane];
                if constexpr (GREEDY) {
                    const int i2 = ti[l * 33 + lane];
                    it = m2 > mt || (m2 == mt && i2 < it) ? i2 : it;
                }
                mt = fmaxf(mt, m2);
            }
#pragma unroll 8
            for (int l = 0; l < 32; ++l) {
                const float m2 = tm[l * 33 + lane], d2 = td[l * 33 + lane];
                if constexpr (GREEDY)
                    dt += ti[l * 33 + lane] == it ? d2 : rescaled_others(d2, m2, mt);
                else
                    dt += rescaled(d2, m2, mt);
            }
            sm[warp - 4][lane] = mt;
            sd[warp - 4][lane] = dt;
            si[warp - 4][lane] = it;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*dead) {
        if (threadIdx.x == 0)
            raise_timeout(a.fail);
        settle_after_failure();
    }
    if (warp == 2)
        tmem_free<1>(tmem, kCols);
    if (static_cast<int>(threadIdx.x) < min(n, kN)) {
        const int per = (n + NG - 1) / NG;
        const int g = static_cast<int>(threadIdx.x) / per, j = static_cast<int>(threadIdx.x) % per;
        float m = sm[4 * g][j], d = sd[4 * g][j];
        int best = si[4 * g][j];
#pragma unroll
        for (int q = 1; q < 4; ++q) {
            const float m2 = sm[4 * g + q][j], d2 = sd[4 * g + q][j];
            if constexpr (GREEDY) {
                best_merge(m, d, best, m2, d2, si[4 * g + q][j]);
            } else {
                const float mn = fmaxf(m, m2);
                d = rescaled(d, m, mn) + rescaled(d2, m2, mn);
                m = mn;
            }
        }
        const int64_t at = threadIdx.x * a.ldp + blockIdx.x;
        if constexpr (GREEDY)
            a.best[at] = make_float4(m, d, __int_as_float(best), 0.f);
        else
            a.part[at] = make_float2(m == -INFINITY ? m : shift_of(m), d);
    }
}

// ---------------------------------------------------------------------------
// the rows that count, in order; their targets, shifts and factors

struct PrepArgs {
    const int64_t *targets;
    int64_t M, V, ignore_index;
    int *n_out;      // targets that are not ignore_index (the divisor of the mean)
    int *rows_out;   // rows listed: those with a target in [0, V)
    unsigned *fail;
    unsigned *done;  // forward: CTAs of the merge that have finished
    int *idx, *tgt;
    int reduction;
    // forward: the values of the rows not listed, and of an empty batch
    float *loss, *row_loss, *lse_out;
    // backward
    const float *lse_in, *grad_scale;
    float *l2, *rs, *alpha;
    unsigned *arrived;  // counters of split tiles
    float head;      // power of two that keeps 16-bit G in range (fp16: 2^14; bf16: 2, so that a factor's
                     // inverse scale is a normal number up to the end of fp32)
};

// What a CTA knows of the listed rows after prep_rows.
struct Listed {
    int rows;
    float inv;  // of a row's own factor: the power of two that it is relative to
};

// By all NT threads of a CTA.  `write`: this CTA writes the call's lists and
// values to memory; s_idx, s_tgt (NULL: not kept) get the list for this CTA.
template <int NT, bool BWD>
__device__ __forceinline__ Listed prep_rows(const PrepArgs &a, bool write, int *s_idx, int *s_tgt)
{
    __shared__ int warp_rows[NT / 32], warp_n[NT / 32];
    __shared__ float warp_max[NT / 32];
    __shared__ int any_bad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0)
        any_bad = 0;
    __syncthreads();
    // each warp owns a contiguous range of rows: counts first, then the list
    const int64_t per = ((a.M + NT - 1) / NT) * 32;
    const int64_t lo = min(per * warp, a.M), hi = min(lo + per, a.M);
    // a factor of the row's own goes into its entries of G; one that all rows share is
    // applied to the sums in fp32, so that an entry of -1 stays one in 16 bits
    const bool own = BWD && a.grad_scale && a.reduction == kReduceNone;
    int rows = 0, n = 0;
    float top = 0.f;
    bool bad = false;
#pragma unroll 8
    for (int64_t i = lo + lane; i < hi; i += 32) {
        const int64_t y = __ldg(a.targets + i);
        if (y != a.ignore_index) {
            ++n;
            if (y >= 0 && y < a.V) {
                ++rows;
                if (own) {
                    const float g = fabsf(__ldg(a.grad_scale + i));
                    top = g > top && g < INFINITY ? g : top;  // NaN and infinity stay in their rows
                }
            } else {
                bad = true;
            }
        }
    }
    if (bad)
        any_bad = 1;
    rows = __reduce_add_sync(0xffffffffu, rows);
    n = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) {
        warp_rows[warp] = rows;
        warp_n[warp] = n;
        warp_max[warp] = top;
    }
    __syncthreads();
    int at = 0;
    Listed list{0, 1.f};
    int n_all = 0;
    top = 0.f;
#pragma unroll 8
    for (int w = 0; w < NT / 32; ++w) {
        at += w < warp ? warp_rows[w] : 0;
        list.rows += warp_rows[w];
        n_all += warp_n[w];
        top = fmaxf(top, warp_max[w]);
    }
    // rows' factors relative to a power of two at or above the largest, so that their
    // 16-bit products with (p - onehot) stay in range whatever the loss scale
    if (BWD) {
        int e = 0;
        if (top > 0.f)
            frexpf(top, &e);
        e = min(max(e, -100), 127);
        list.inv = ldexpf(a.head, -e);
        if (write && threadIdx.x == 0)
            *a.alpha = (a.reduction == kReduceMean ? 1.f / static_cast<float>(max(n_all, 1)) : 1.f) *
                       // no row: zeros, which a factor of NaN must not touch
                       (a.grad_scale && !own && list.rows ? __ldg(a.grad_scale) : 1.f) * ldexpf(1.f / a.head, e);
        if (write)
            for (int i = threadIdx.x; i < kSplitCounters; i += NT)
                a.arrived[i] = 0u;
    }
    if (write && threadIdx.x == 0) {
        *a.n_out = n_all;
        *a.rows_out = list.rows;
        *a.fail = 0u;
        *a.done = 0u;
        if (any_bad)
            atomicOr(&g_flags, kFlagBadTarget);
        if (!BWD && a.M == 0 && a.reduction != kReduceNone)
            *a.loss = a.reduction == kReduceMean ? __int_as_float(0x7fc00000) : 0.f;
    }
    // four rounds' loads ahead of any of their stores
    constexpr int R = 4;
#pragma unroll 1
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * R) {
        int64_t y[R];
        float lse[R], g[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t i = i0 + 32 * r + lane;
            y[r] = i < hi ? __ldg(a.targets + i) : a.ignore_index;
            lse[r] = BWD && write && i < hi ? __ldg(a.lse_in + i) : 0.f;
            g[r] = own && write && i < hi ? __ldg(a.grad_scale + i) : 1.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t i = i0 + 32 * r + lane;
            const bool skip = y[r] == a.ignore_index;
            const bool listed = !skip && y[r] >= 0 && y[r] < a.V;
            const unsigned votes = __ballot_sync(0xffffffffu, listed);
            if (listed) {
                const int pos = at + __popc(votes & ((1u << lane) - 1));
                if (s_idx) {
                    s_idx[pos] = static_cast<int>(i);
                    s_tgt[pos] = static_cast<int>(y[r]);
                }
                if (write) {
                    a.idx[pos] = static_cast<int>(i);
                    a.tgt[pos] = static_cast<int>(y[r]);
                    if (BWD) {
                        a.l2[pos] = lse[r] * kLog2e;
                        a.rs[pos] = g[r] * list.inv;
                    }
                }
            } else if (!BWD && write && i < hi) {
                const float v = skip ? 0.f : __int_as_float(0x7fc00000);
                a.row_loss[i] = v;
                if (a.lse_out)
                    a.lse_out[i] = v;
            }
            at += __popc(votes);
        }
    }
    return list;
}

// sum_k a[k] b[k] of two rows in fp32, by NT threads (a warp's share in each of its lanes).
template <typename T, int NT>
__device__ __forceinline__ float row_dot(const T *a, const T *b, int64_t K, bool vec)
{
    const int lane = threadIdx.x & (NT - 1);
    float s0 = 0.f, s1 = 0.f;
    int64_t k = 0;
    if (vec) {
#pragma unroll 4
        for (int64_t j = lane; j < K / 8; j += NT) {
            float x[8], y[8];
            Elem<T>::unpack(reinterpret_cast<const uint4 *>(a)[j], x);
            Elem<T>::unpack(reinterpret_cast<const uint4 *>(b)[j], y);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                s0 = fmaf(x[i], y[i], s0);
                s1 = fmaf(x[i + 1], y[i + 1], s1);
            }
        }
        k = K / 8 * 8;
    }
    for (int64_t j = k + lane; j < K; j += NT)
        s0 = fmaf(Elem<T>::load(a + j), Elem<T>::load(b + j), s0);
    return warp_sum(s0 + s1);
}

// Packed copy of the listed rows (dst [.., lds], zeros in columns K .. lds and in
// the rows up to the next multiple of `pad`), the logits of their targets, and
// zeros in the rows of `zero` that are not listed.  One warp per row.
struct GatherArgs {
    const void *src;
    int64_t ss;
    void *dst;
    int64_t lds;
    int64_t K;
    int pad;
    int vec;            // src allows 16-byte loads
    // targets' logits, or (backward) the rows' losses in their place
    const void *w;      // NULL: none
    int64_t ws;
    int wvec;           // w and src allow 16-byte loads
    float *xy;          // forward: x_y
    float *gy;          // backward: (p_y - 1) times the row's factor
    // backward: unlisted rows of the hidden gradient
    void *zero;
    int64_t zs;
    int zvec;           // zero allows 16-byte stores
    int64_t M, V, ignore_index;
    const int64_t *targets;
    const float *row_loss;  // NULL: none given
};

// The 16 bytes that begin `off` (even, < 16) bytes into the aligned v[0], v[1].
__device__ __forceinline__ uint4 shifted_vector(const uint4 *v, int off)
{
    const uint4 a = __ldg(v), b = __ldg(v + 1);
    uint32_t x[5] = {a.x, a.y, a.z, a.w, b.x};
    if (off & 8) {
        x[0] = a.z, x[1] = a.w, x[2] = b.x, x[3] = b.y, x[4] = b.z;
        if (off & 4)
            x[0] = a.w, x[1] = b.x, x[2] = b.y, x[3] = b.z, x[4] = b.w;
    } else if (off & 4) {
        x[0] = a.y, x[1] = a.z, x[2] = a.w, x[3] = b.x, x[4] = b.y;
    }
    if (off & 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = __funnelshift_r(x[i], x[i + 1], 16);
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// By one warp of `step`; row_of(i), target_of(i) and (backward) lse_of(i) of the n
// listed rows, entry_of(i, ln p_y) the backward's entry of its target.
template <typename T, typename RowOf, typename TargetOf, typename LseOf, typename EntryOf>
__device__ __forceinline__ void gather_rows(const GatherArgs &a, int64_t n, int64_t first, int64_t step,
                                            RowOf row_of, TargetOf target_of, LseOf lse_of, EntryOf entry_of)
{
    const int lane = threadIdx.x & 31;
    const int64_t rows = (n + a.pad - 1) / a.pad * a.pad;
    const T zero_value = T(0.f);
    for (int64_t i = first; i < rows; i += step) {
        T *d = static_cast<T *>(a.dst) + i * a.lds;
        if (i >= n) {
            for (int64_t j = lane; j < a.lds / 8; j += 32)
                reinterpret_cast<uint4 *>(d)[j] = make_uint4(0, 0, 0, 0);
            continue;
        }
        const T *s = static_cast<const T *>(a.src) + row_of(i) * a.ss;
        // on its way while the row is copied
        const float known = a.row_loss ? __ldg(a.row_loss + row_of(i)) : a.gy ? lse_of(i) : 0.f;
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(s) & 15);
        const uint4 *s0 = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(s) - off);
        int64_t done = 0;
        if (a.vec) {  // K may end inside the last vector: the rest is zeroed one by one
            done = a.K / 8 * 8;
#pragma unroll 4
            for (int64_t j = lane; j < a.K / 8; j += 32)
                reinterpret_cast<uint4 *>(d)[j] = __ldg(reinterpret_cast<const uint4 *>(s) + j);
        }
#pragma unroll 2
        for (int64_t j = done / 8 + lane; j < a.lds / 8; j += 32) {
            if (16 * (j + 2) <= off + 2 * a.K && (j > 0 || off == 0)) {
                reinterpret_cast<uint4 *>(d)[j] = shifted_vector(s0 + j, off);
                continue;
            }
            alignas(16) T v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = 8 * j + i < a.K ? s[8 * j + i] : zero_value;
            reinterpret_cast<uint4 *>(d)[j] = *reinterpret_cast<const uint4 *>(v);
        }
        if (a.w) {
            const float x = row_dot<T, 32>(s, static_cast<const T *>(a.w) + target_of(i) * a.ws, a.K, a.wvec);
            if (lane == 0) {
                if (a.xy)
                    a.xy[i] = x;
                else
                    a.gy[i] = entry_of(i, x - known);
            }
        } else if (a.row_loss && lane == 0) {
            a.gy[i] = entry_of(i, -known);
        }
    }
    if (a.zero)
        for (int64_t i = first; i < a.M; i += step) {
            const int64_t y = a.targets[i];
            if (y != a.ignore_index && y >= 0 && y < a.V)
                continue;
            T *z = static_cast<T *>(a.zero) + i * a.zs;
            const int64_t whole = a.zvec ? a.K / 8 : 0;
            for (int64_t j = lane; j < whole; j += 32)
                reinterpret_cast<uint4 *>(z)[j] = make_uint4(0, 0, 0, 0);
            for (int64_t j = whole * 8 + lane; j < a.K; j += 32)
                z[j] = zero_value;
        }
}

constexpr int kFewRows = 64;  // rows that skinny_kernel takes

// Many rows: one CTA lists them, then many pack them.
template <int NT, bool BWD>
__global__ void __launch_bounds__(NT) lin_prep_kernel(const PrepArgs a)
{
    next_kernel_may_start();
    prep_rows<NT, BWD>(a, true, nullptr, nullptr);
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT) lin_gather_kernel(const GatherArgs a, const PrepArgs p)
{
    next_kernel_may_start();
    wait_prerequisite_grid();
    gather_rows<T>(
        a, *p.rows_out, blockIdx.x * int64_t{NT / 32} + (threadIdx.x >> 5), gridDim.x * int64_t{NT / 32},
        [&](int64_t i) { return int64_t{p.idx[i]}; }, [&](int64_t i) { return int64_t{p.tgt[i]}; },
        [&](int64_t i) { return p.lse_in[p.idx[i]]; }, [&](int64_t i, float lnp) { return expm1f(lnp) * p.rs[i]; });
}

// Up to kStartRows rows: every CTA lists them for itself (8 KB of targets from
// L2) and packs its own, one launch in place of two.
constexpr int kStartRows = 1024;

template <typename T, bool BWD, int NT>
__global__ void __launch_bounds__(NT) lin_start_kernel(const GatherArgs a, const PrepArgs p)
{
    __shared__ int idx[kStartRows], tgt[kStartRows];
    next_kernel_may_start();
    const Listed list = prep_rows<NT, BWD>(p, blockIdx.x == 0, idx, tgt);
    __syncthreads();
    gather_rows<T>(
        a, list.rows, blockIdx.x * int64_t{NT / 32} + (threadIdx.x >> 5), gridDim.x * int64_t{NT / 32},
        [&](int64_t i) { return int64_t{idx[i]}; }, [&](int64_t i) { return int64_t{tgt[i]}; },
        [&](int64_t i) { return p.lse_in[idx[i]]; },
        [&](int64_t i, float lnp) {
            const float g = p.grad_scale && p.reduction == kReduceNone ? p.grad_scale[idx[i]] : 1.f;
            return expm1f(lnp) * (g * list.inv);
        });
}

// Rows as they stand (weights, or hidden states of the arg max, that a tensor map cannot read).
template <typename T, int NT>
__global__ void __launch_bounds__(NT) lin_pack_kernel(const GatherArgs a, int64_t n)
{
    next_kernel_may_start();
    wait_prerequisite_grid();
    gather_rows<T>(
        a, n, blockIdx.x * int64_t{NT / 32} + (threadIdx.x >> 5), gridDim.x * int64_t{NT / 32},
        [](int64_t i) { return i; }, [](int64_t) { return int64_t{0}; }, [](int64_t) { return 0.f; },
        [](int64_t, float) { return 0.f; });
}

// ---------------------------------------------------------------------------
// the partial pairs of each row, merged in order

struct MergeArgs {
    const float2 *part;
    const float4 *best;
    int parts;
    const int *n_ptr;
    int n_host;
    const int *idx;
    const float *xy;
    float *row_loss, *lse;
    float *loss;        // NULL: no reduction
    const int *n_mean;  // targets that are not ignored
    const unsigned *fail;
    unsigned *done;
    int64_t M;
    int reduction;
    // arg max: its logit is formed again from these rows
    int64_t *token;
    float *logprob;
    const void *h, *w;
    int64_t hs, ws, K, V;
    int vec;
};

// ln(1 + others / e^x_y) for the others' sum d about the shift s (-inf: none),
// and ln(others + e^x_y).
__device__ __forceinline__ float loss_beside(float s, float d, float xy, float &lse)
{
    lse = __int_as_float(0x7fc00000);
    if (!(xy < INFINITY))
        return lse;
    if (s == -INFINITY && d == 0.f) {  // the only class
        lse = xy;
        return xy - xy;
    }
    const float shift = s == -INFINITY ? 0.f : s;
    const float t = fmaf(xy, kLog2e, -shift);  // log2 of e^x_y about the shift
    if (t > -20.f) {
        const float loss = log1pf(d * exp2f(-t));
        lse = xy + loss;
        return loss;
    }
    // an unlikely target: others / e^x_y might overflow
    const float l = logf(d + exp2f(t));
    lse = fmaf(shift, kLn2, l);
    return l - t * kLn2;
}

// One warp per listed row; the last CTA to finish adds the row losses in an
// order fixed by M.
template <int NT>
__global__ void __launch_bounds__(NT) lin_merge_kernel(const MergeArgs a)
{
    __shared__ int last;
    const int lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x * int64_t{NT / 32} + (threadIdx.x >> 5);
    next_kernel_may_start();
    wait_prerequisite_grid();
    if (row < *a.n_ptr) {
        const float2 *part = a.part + row * a.parts;
        float s = -INFINITY, d = 0.f;
#pragma unroll 4
        for (int p = lane; p < a.parts; p += 32) {
            const float2 q = part[p];
            const float sn = fmaxf(s, q.x);
            d = shifted(d, s, sn) + shifted(q.y, q.x, sn);
            s = sn;
        }
        float top = s;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        d = warp_sum(shifted(d, s, top));
        if (lane == 0) {
            const int64_t out = a.idx[row];
            float lse;
            a.row_loss[out] = loss_beside(top, d, a.xy[row], lse);
            if (a.lse)
                a.lse[out] = lse;
        }
    }
    if (!a.loss)
        return;
    __threadfence();
    __syncthreads();
    if (gridDim.x > 1) {
        if (threadIdx.x == 0)
            last = atomicAdd(a.done, 1u) == gridDim.x - 1;
        __syncthreads();
        if (!last)
            return;
        __threadfence();
    }
    const float s = sum_row_losses<NT>(a.row_loss, a.M, threadIdx.x, 1);
    if (threadIdx.x == 0)
        *a.loss = __ldcg(a.fail) ? __int_as_float(0x7fc00000)
                                 : a.reduction == kReduceMean ? s / static_cast<float>(*a.n_mean) : s;
}

// Up to 64 rows as they stand, none listed or packed before: one CTA merges their
// partials, forms their targets' logits and the mean.
template <typename T, int NT>
__global__ void __launch_bounds__(NT) lin_few_kernel(const MergeArgs a, const PrepArgs p)
{
    __shared__ int n_all, any_bad;
    const int lane = threadIdx.x & 31;
    next_kernel_may_start();
    if (threadIdx.x == 0)
        n_all = any_bad = 0;
    __syncthreads();
    // the dot products read nothing that the kernel before wrote
    constexpr int kMost = (kFewRows + NT / 32 - 1) / (NT / 32);
    float xy[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        const int64_t row = (threadIdx.x >> 5) + k * (NT / 32);
        xy[k] = 0.f;
        if (row >= a.M)
            continue;
        const int64_t y = p.targets[row];
        if (y == p.ignore_index)
            continue;
        const bool good = y >= 0 && y < p.V;
        if (good)
            xy[k] = row_dot<T, 32>(static_cast<const T *>(a.h) + row * a.hs, static_cast<const T *>(a.w) + y * a.ws,
                                   a.K, a.vec);
        if (lane == 0) {
            atomicAdd(&n_all, 1);
            if (!good)
                any_bad = 1;
        }
    }
    wait_prerequisite_grid();
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        const int64_t row = (threadIdx.x >> 5) + k * (NT / 32);
        if (row >= a.M)
            continue;
        const int64_t y = p.targets[row];
        const float2 *part = a.part + row * a.parts;
        float s = -INFINITY, d = 0.f;
#pragma unroll 4
        for (int q = lane; q < a.parts; q += 32) {
            const float2 v = part[q];
            const float sn = fmaxf(s, v.x);
            d = shifted(d, s, sn) + shifted(v.y, v.x, sn);
            s = sn;
        }
        float top = s;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        d = warp_sum(shifted(d, s, top));
        if (lane == 0) {
            float lse = y == p.ignore_index ? 0.f : __int_as_float(0x7fc00000), loss = lse;
            if (y != p.ignore_index && y >= 0 && y < p.V)
                loss = loss_beside(top, d, xy[k], lse);
            a.row_loss[row] = loss;
            if (a.lse)
                a.lse[row] = lse;
        }
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0 && any_bad)
        atomicOr(&g_flags, kFlagBadTarget);
    if (!a.loss)
        return;
    const float s = sum_row_losses<NT>(a.row_loss, a.M, threadIdx.x, 1);
    if (threadIdx.x == 0)
        *a.loss = __ldcg(a.fail) ? __int_as_float(0x7fc00000)
                                 : a.reduction == kReduceMean ? s / static_cast<float>(n_all) : s;
}

// One CTA per row: its partials, then the dot product of its token.
template <typename T, int NT>
__global__ void __launch_bounds__(NT) lin_token_kernel(const MergeArgs a)
{
    __shared__ float sm[NT / 32], sd[NT / 32];
    __shared__ int si[NT / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    next_kernel_may_start();
    wait_prerequisite_grid();
    const float4 *part = a.best + row * a.parts;
    float m = -INFINITY, d = 0.f;
    int best = INT32_MAX;
#pragma unroll 2
    for (int p = threadIdx.x; p < a.parts; p += NT) {
        const float4 q = part[p];
        best_merge(m, d, best, q.x, q.y, __float_as_int(q.z));
    }
    float mt = m;
    int it = best;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, mt, off);
        const int i2 = __shfl_xor_sync(0xffffffffu, it, off);
        if (m2 > mt || (m2 == mt && i2 < it)) {
            mt = m2;
            it = i2;
        }
    }
    d = warp_sum(best == it ? d : rescaled_others(d, m, mt));
    if (lane == 0) {
        sm[warp] = mt;
        sd[warp] = d;
        si[warp] = it;
    }
    __syncthreads();
    m = sm[0];
    d = sd[0];
    best = si[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w)
        best_merge(m, d, best, sm[w], sd[w], si[w]);
    // no index: nothing but NaN or -inf, or partials that a kernel which gave up
    // on a copy left unwritten (any bits: the index is checked before it is used)
    float lse, lp = __int_as_float(0x7fc00000);
    const bool found = best >= 0 && best < a.V;
    if (found) {
        const float x = row_dot<T, NT>(static_cast<const T *>(a.h) + row * a.hs,
                                       static_cast<const T *>(a.w) + best * a.ws, a.K, a.vec);
        __syncthreads();
        if (lane == 0)
            sm[warp] = x;
        __syncthreads();
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w)
            sum += sm[w];
        lp = -loss_beside(shift_of(m), d, sum, lse);
    }
    if (threadIdx.x == 0) {
        a.token[row] = found ? best : 0;
        a.logprob[row] = lp;
    }
}

}  // namespace gbce
