// mpt_xent.cu -- softmax cross entropy of a linear head over a large
// vocabulary, with its loss-scaled gradients (mpt_xent of include/mpt.h).
//
//   z = H W^T            H: n x d activations, W: v x d head, 16-bit
//   loss_i = log(1 + sum_{u != t} exp(z_u - z_t)),  t = target of row i
//   dz_iu  = exp(z_iu - lse_i) - [u = t]            (at u = t: expm1(-loss_i))
//   dH = g dz W,  dW = g dz^T H,  g = S / valid rows (or S)
//
// No buffer holds all logits of a large call.  The forward pass reduces each
// 256-column tile of z to a maximum and a sum per row while the next tile is
// multiplied; the backward pass goes through the vocabulary in pieces: multiply
// z again, write dz of the piece in 16 bits, and multiply it with W (dH, summed
// over the pieces in binary32) and with H (this piece's rows of dW, final at
// once).  More than 16384 rows are cut, too, and a piece's dW is then summed in
// binary32 over the cuts.  Where all of a call's logits fit in a buffer of their
// own and moving them is cheaper than multiplying again, they stay there between
// the passes.
//
// The loss is formed from the other columns' sum against the target's logit,
// so a sure answer's small loss keeps its digits, and dz at the target comes
// from the loss for the same reason.  dz is rounded to 16 bits once, scaled
// by 2^15 in binary16 so that probabilities down to 2^-29 keep full
// precision; the loss scale and 1/n are applied to the binary32 sums.
//
// All four products run on the tensor cores in one kernel: one CTA per SM,
// one warp that loads tiles by TMA, one that issues the products, eight
// warps that turn finished accumulators into results; two accumulators in
// tensor memory let the products of a tile run under the results of the last.
// Two CTAs share a tile of 256 x 256 (each loads half of either operand, so
// an operand byte feeds twice the products); for at most 128 rows every CTA
// works alone on 128 x 256.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/mpt.h"
#include "sm100.cuh"

namespace {

using namespace sm100;

constexpr int kRows = 128;              // of a CTA's tile
constexpr int kTileN = 256, kTileK = 64;
constexpr int kResultWarps = 8, kThreads = 32 * (kResultWarps + 2);  // then one that loads, one that multiplies
constexpr int kBytesA = kRows * kTileK * 2;
constexpr int kHalf = kTileN / 2;       // columns of one result warp
// The tensor cores drop what lies below an accumulator's last place, 16 of K
// at a time: 1e-7 of the sum each time where the terms have one sign, always
// downwards.  Logits are therefore taken out after 512 of K and added with
// rounding to nearest (losses of 509 x 50257 x 2048 2e-6 off without, 1e-7
// with, the target's logit formed apart), in the backward pass as in the
// forward pass: a logit that is multiplied again has to be the one that its
// row's sum of exponentials was made from.  (Logits of 1000 to 2000, 4096 and
// 8192 wide, gave gradients 10% and 38% off where the backward pass did not.)
// What stays is 2.4e-6 of a logit whose products have one sign: 0.005 of the loss
// at logits of 2000, where the logits' sum in binary32 to nearest leaves 0.002.
constexpr int kPromote = 512 / kTileK;

// Results leave through shared memory: each half of the result warps has one
// box of 128 rows of 128 bytes, which TMA stores.  (With rows stored straight
// from registers, 16 bytes of 32 rows at a time, and tiles in plain order, the
// gradients of 1001 x 50257 x 1024 took 423 us; with both changed 361.)
constexpr int kOutBytes = kRows * 128;

// Shared memory of one load stage, and how many fit.  Seven stages keep
// 224 KB of loads in flight (the forward pass stores nothing by TMA).
template <bool kPair, int kMode> struct Shape {
    static constexpr int kBytesB = (kPair ? kTileN / 2 : kTileN) * kTileK * 2;
    static constexpr int kStageBytes = kBytesA + kBytesB;
    static constexpr int kOut = kMode == 0 ? 0 : 2 * kOutBytes;
    static constexpr int kStages = (7 * 32768 - kOut) / kStageBytes;
    static constexpr int kSmem = kStages * kStageBytes + kOut + 1024;
    static constexpr int kTileM = kPair ? 2 * kRows : kRows;
    static constexpr int kCtas = kPair ? 2 : 1;
};
constexpr int kMaxCtas = 148;
constexpr float kLog2e = 1.4426950408889634f;
constexpr size_t kAlign = 256;

enum Mode { kLoss, kDz, kGrad };  // the places of MPT_XENT_PASS_*

// One product: mt x nt output tiles, each summed over kb blocks of 64, the
// sum cut into `splits` parts.  Tiles are taken in bands of `band` rows of
// tiles, the rows of a band first: what runs at the same time then shares
// the band's rows of A, held in L2, and few columns of B.  band 1: along a row.
struct Job {
    int32_t mt, nt, splits, kb;
    int32_t band;
    int32_t tn;           // columns of a tile: a multiple of 16, at most 256
    uint32_t idesc;
    int32_t tiles;
    int32_t is_dw;        // kGrad: dW (else dH)
    // kGrad: results are final, g * sum in 16 bits (else binary32 sums)
    int32_t final;
    int32_t add;          // to the sums that are there
    int32_t rows;
    int32_t wide;         // TMA can store them; if not:
    uint16_t* to;
    int64_t ld;
};

// Start of the workspace.
struct Control {
    float gscale;           // S / rows, with the scaling of dz taken back
    unsigned int ticket;    // of the merging CTAs
    int32_t status[kMaxCtas];  // of the forward pass's CTAs: 1 after a wait that ran out
};

struct RowStats {
    const float* lse;
    const float* loss;
};

struct GemmArgs {
    CUtensorMap a[2], b[2], out[2];
    Job job[2];           // kGrad: dH and dW, the longer tiles first
    // Tile order, worked out by every worker alone: the first job's tiles go
    // round; `late` workers have one more of them, while they are at it the
    // others take `ahead` rounds of the second job; then all go round.
    int32_t late, ahead;
    // rows and columns of the logits
    int32_t n, v;
    const void* targets;
    int32_t target_bytes;
    int64_t ignore;
    // kLoss
    float2* part;         // [n][part_ld]: maximum and sum of half a tile's columns
    int32_t part_ld;
    Control* control;
    float* z;             // [n][z_ld]: the logits, where a call keeps them
    int64_t z_ld;
    // kDz
    RowStats stats;
    int32_t col0;         // first column of the piece
    float exponent;       // dz is scaled by 2^exponent
    // kGrad
    int32_t d;
    float* poison;        // kDz, kGrad: the loss, NaN after a wait that ran out
    int32_t give_up;      // test hook: each block gives up after its first loads
};

__device__ __forceinline__ int64_t target_of(const GemmArgs& g, int row)
{
    return g.target_bytes == 8 ? static_cast<const int64_t*>(g.targets)[row]
                               : (int64_t)static_cast<const int32_t*>(g.targets)[row];
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float x, float y)
{
    if constexpr (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

struct Tile {
    int job, m, n, split, kb0, kb1, tn;
};

// The k-th tile of a worker, or -1.
__device__ __forceinline__ int tile_number(const GemmArgs& g, int worker, int workers, int k)
{
    const int first = g.job[0].tiles, second = g.job[1].tiles;
    if (worker + k * workers < first)
        return worker + k * workers;
    if (second == 0)
        return -1;
    const bool late = worker < g.late;
    const int j = k - (first / workers + (late ? 1 : 0));
    const int early = workers - g.late, base = g.ahead * early;
    const int i = late ? base + j * workers + worker
                       : j < g.ahead ? j * early + worker - g.late : base + (j - g.ahead) * workers + worker;
    return i < second ? first + i : -1;
}

__device__ __forceinline__ Tile tile_at(const GemmArgs& g, int t)
{
    Tile r;
    r.job = t >= g.job[0].tiles ? 1 : 0;
    const Job& j = g.job[r.job];
    int i = t - (r.job ? g.job[0].tiles : 0);
    r.split = 0;
    r.tn = j.tn;
    if (j.splits > 1) {
        r.split = i / (j.mt * j.nt);
        i -= r.split * (j.mt * j.nt);
    }
    if (j.band == 1) {
        r.m = i / j.nt;
        r.n = i - r.m * j.nt;
    } else {
        const int m0 = i / (j.band * j.nt) * j.band, rows = min(j.band, j.mt - m0);
        i -= m0 * j.nt;
        r.n = i / rows;
        r.m = m0 + i - r.n * rows;
    }
    r.kb0 = 0;
    r.kb1 = j.kb;
    if (j.splits > 1) {
        r.kb0 = (int)((int64_t)j.kb * r.split / j.splits);
        r.kb1 = (int)((int64_t)j.kb * (r.split + 1) / j.splits);
    }
    return r;
}

__device__ __forceinline__ bool next_tile(const GemmArgs& g, int worker, int workers, int k, Tile& u)
{
    const int t = tile_number(g, worker, workers, k);
    if (t >= 0)
        u = tile_at(g, t);
    return t >= 0;
}

// ---------------------------------------------------------------------------
// results: one thread per row and half of the tile's columns
// ---------------------------------------------------------------------------

// What a result thread has to know of its row; read before the accumulator is
// waited for.
struct Row {
    int64_t target;       // -1 beyond the last row
    float lse, loss;      // kDz
};

template <int kMode>
__device__ __forceinline__ Row row_at(const GemmArgs& g, int row)
{
    Row r{-1, 0.0f, 0.0f};
    if (kMode != kGrad && row < g.n) {
        r.target = target_of(g, row);
        if (kMode == kDz) {
            r.lse = g.stats.lse[row];
            r.loss = g.stats.loss[row];
        }
    }
    return r;
}

// The target's column among `width` ones from col0 on, or -1.
__device__ __forceinline__ int hit_at(const GemmArgs& g, int64_t target, int col0, int width)
{
    if (target < 0 || target >= g.v || target == g.ignore)
        return -1;
    const int h = (int)target - col0;
    return h >= 0 && h < width ? h : -1;
}

// Maximum and sum of exponentials of `width` columns; the target's column is
// left out.
__device__ __forceinline__ void rows_loss(const GemmArgs& g, int part, int col0, int width, int row, const Row& me,
                                          float (&z)[kHalf])
{
    const int hit = hit_at(g, me.target, col0, width);
    const int cols = min(width, g.v - col0);
    if (g.z && row < g.n) {
        float* to = g.z + (int64_t)row * g.z_ld + col0;
#pragma unroll
        for (int k = 0; k < kHalf; k += 8)
            if (k < width)
                store32(to + k, z + k);
    }
    if (cols < kHalf) {
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            z[k] = k < cols ? z[k] : -INFINITY;
    }
    if (__any_sync(0xffffffffu, hit >= 0)) {
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            z[k] = k == hit ? -INFINITY : z[k];
    }
    float m4[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
    for (int k = 4; k < kHalf; ++k)
        m4[k & 3] = fmaxf(m4[k & 3], z[k]);
    const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
    // a row of nothing but -inf sums to zero: no inf - inf
    const float base = top == -INFINITY ? 0.0f : top * kLog2e;
    const uint64_t scale2 = pair_of(kLog2e, kLog2e), base2 = pair_of(-base, -base);
    uint64_t s4[4] = {};
#pragma unroll
    for (int c = 0; c < kHalf; c += 16) {
        if (c < cols) {
#pragma unroll
            for (int k = c; k < c + 16; k += 2) {
                const float2 e = of_pair(fma2(pair_of(z[k], z[k + 1]), scale2, base2));
                s4[(k / 2) & 3] = add2(s4[(k / 2) & 3], pair_of(exp2_fast(e.x), exp2_fast(e.y)));
            }
        }
    }
    const float2 sum = of_pair(add2(add2(s4[0], s4[1]), add2(s4[2], s4[3])));
    if (row < g.n)
        g.part[(int64_t)row * g.part_ld + part] = make_float2(top, sum.x + sum.y);
}

// A result warp's place in its half's box: rows of 128 bytes, the 16-byte
// pieces of a row exchanged as TMA's 128-byte swizzle does.
struct Box {
    uint32_t row_at;      // this thread's row
    uint32_t at;
    int row, half;
    bool first;           // of the half's threads: it stores

    __device__ __forceinline__ void put(int piece, uint32_t a, uint32_t b, uint32_t c, uint32_t d) const
    {
        shared_store16(row_at + ((piece ^ (row & 7)) << 4), a, b, c, d);
    }
    // before the first put: the last store has read the box
    __device__ __forceinline__ void open() const
    {
        if (first)
            store_wait_read();
        named_sync(1 + half, 32 * kResultWarps / 2);
    }
    // after the last put; the first thread then stores and commits
    __device__ __forceinline__ void close() const
    {
        fence_async();
        named_sync(1 + half, 32 * kResultWarps / 2);
    }
};

// dz of 128 columns, rounded to 16 bits once.
template <bool kBf16>
__device__ __forceinline__ void rows_dz(const GemmArgs& g, int col0, int width, int row0, const Row& me,
                                        float (&z)[kHalf], const Box& box)
{
    const int cols = min(width, g.v - g.col0 - col0);  // col0 counts inside the piece
    const int hit = hit_at(g, me.target, g.col0 + col0, width);
    const bool live = row0 + box.row < g.n && me.target != g.ignore;
    const bool edge = cols < width || !__all_sync(0xffffffffu, live);
    const float base = fmaf(-me.lse, kLog2e, g.exponent);
    const uint64_t scale2 = pair_of(kLog2e, kLog2e), base2 = pair_of(base, base);
#pragma unroll
    for (int c = 0; c < kHalf; c += 64) {
        if (c >= width)
            break;
        const bool hits = __any_sync(0xffffffffu, hit >= c && hit < c + 64);
#pragma unroll
        for (int k = c; k < c + 64; k += 2) {
            const float2 e = of_pair(fma2(pair_of(z[k], z[k + 1]), scale2, base2));
            z[k] = exp2_fast(e.x);
            z[k + 1] = exp2_fast(e.y);
        }
        if (edge) {
#pragma unroll
            for (int k = c; k < c + 64; ++k)
                z[k] = live && k < cols ? z[k] : 0.0f;
        }
        if (hits) {
            const float at_target = ldexpf(expm1f(-me.loss), (int)g.exponent);
#pragma unroll
            for (int k = c; k < c + 64; ++k)
                z[k] = k == hit ? at_target : z[k];
        }
        uint32_t o[32];
#pragma unroll
        for (int k = 0; k < 32; ++k)
            o[k] = pack2<kBf16>(z[c + 2 * k], z[c + 2 * k + 1]);
        box.open();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            box.put(k, o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        box.close();
        if (box.first) {
            if (c < cols && row0 < g.n)
                tma_store(&g.out[0], box.at, col0 + c, row0);
            store_commit();
        }
    }
}

// 128 columns of a gradient's binary32 sums.
__device__ __forceinline__ void rows_sums(const GemmArgs& g, const Job& j, const CUtensorMap* out, int split, int col0,
                                          int width, int row0, uint32_t tmem, const Box& box)
{
#pragma unroll 1
    for (int c = 0; c < width; c += 32) {
        if (col0 + c >= g.d)
            break;
        __syncwarp();
        uint32_t r[32];
        tmem_load32(tmem + c, r);
        tmem_wait_load(r);
        box.open();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            box.put(k, r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
        box.close();
        if (box.first && row0 < j.rows) {
            if (j.add)
                tma_store3<true>(out, box.at, col0 + c, row0, split);
            else
                tma_store3<false>(out, box.at, col0 + c, row0, split);
            store_commit();
        }
    }
}

// 128 columns of a gradient, final.
template <bool kBf16>
__device__ __forceinline__ void rows_final(const GemmArgs& g, const Job& j, const CUtensorMap* out, int col0, int width, int row0,
                                           uint32_t tmem, const Box& box)
{
    const float scale = g.control->gscale;
    const int row = row0 + box.row;
#pragma unroll 1
    for (int c = 0; c < width; c += 64) {
        if (col0 + c >= g.d)
            break;
        __syncwarp();
        uint32_t r[2][32], o[32];
        tmem_load32(tmem + c, r[0]);
        tmem_load32(tmem + c + 32, r[1]);
        tmem_wait_load(r[0]);
        tmem_wait_load(r[1]);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const float* z = reinterpret_cast<const float*>(r[e / 16]) + 2 * (e % 16);
            o[e] = pack2<kBf16>(z[0] * scale, z[1] * scale);
        }
        if (j.wide) {
            box.open();
#pragma unroll
            for (int k = 0; k < 8; ++k)
                box.put(k, o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else if (row < j.rows) {
            uint16_t* to = j.to + (int64_t)row * j.ld + col0 + c;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                if (col0 + c + 2 * e < g.d) {
                    to[2 * e] = (uint16_t)(o[e] & 0xFFFFu);
                    to[2 * e + 1] = (uint16_t)(o[e] >> 16);
                }
            }
        }
        if (j.wide) {
            box.close();
            if (box.first && row0 < j.rows) {
                tma_store(out, box.at, col0 + c, row0);
                store_commit();
            }
        }
    }
}

// ---------------------------------------------------------------------------
// the product kernel
// ---------------------------------------------------------------------------

constexpr uint32_t kBlock = 64 * kTileK * 2;  // of 64 M or N elements of an MN-major tile

// Place in a ring of load stages.
template <int kStages> struct Ring {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++at == kStages) {
            at = 0;
            phase ^= 1;
        }
    }
};

template <bool kValue> struct Flag {
    static constexpr bool value = kValue;
};

// f(A is MN-major, B is MN-major) of the job: logits are rows times rows, dH
// is dz's rows times W's columns, dW dz's columns times H's columns.
template <int kMode, class F>
__device__ __forceinline__ void by_layout(bool dw, F&& f)
{
    if constexpr (kMode != kGrad)
        f(Flag<false>{}, Flag<false>{});
    else if (!dw)
        f(Flag<false>{}, Flag<true>{});
    else
        f(Flag<true>{}, Flag<true>{});
}

// After a wait that ran out: wait (bounded) until every load that was issued has
// landed, in either CTA of a pair; both signal the first one's barriers, which
// alone expects their bytes.  steps0 and steps1 are the loads that the CTAs have
// issued: no more than a ring apart, since a stage is loaded again only after
// both its halves were multiplied.  Where one CTA is ahead the first makes up for
// the other: it expects what only its pair has loaded, and counts what its pair
// never will as landed.
template <bool kPair, int kStages>
__device__ __forceinline__ void drain_loads(uint32_t full, uint32_t steps0, uint32_t steps1, uint32_t bytes, int lane)
{
    const uint32_t most = max(steps0, steps1);
    for (uint32_t b = most > kStages ? most - kStages : 0; b < most; ++b) {
        const uint32_t bar = full + (b % kStages) * 8;
        if (lane == 0) {
            if (kPair && b >= steps0)
                mbar_expect(bar, bytes);
            if (kPair && b >= steps1)
                mbar_landed(bar, bytes);
        }
        __syncwarp();
        mbar_wait(bar, (b / kStages) & 1, nullptr);
    }
}

// After a wait that ran out a block's tiles may be missing: NaN goes where they
// are, or into what everything else is made from, so that neither a loss nor a
// gradient that is not whole looks like one that is (an optimizer step sees the
// gradients only).  The block's own stores are done.
template <int kTileM, int kMode>
__device__ __forceinline__ void poison_results(const GemmArgs& g, int worker, int workers, uint32_t rank)
{
    const float nan = __int_as_float(0x7fc00000);
    if (kMode != kLoss && threadIdx.x == 0) {
        *g.poison = nan;
        g.control->gscale = nan;  // sums that are not rounded yet, later pieces
    }
    for (int k = 0, t; (t = tile_number(g, worker, workers, k)) >= 0; ++k) {
        const Tile u = tile_at(g, t);
        const int row0 = u.m * kTileM + (int)rank * kRows;
        if constexpr (kMode == kLoss) {
            const int row = row0 + (int)threadIdx.x % kRows, half = (int)threadIdx.x / kRows;
            if (half < 2 && row < g.n)
                g.part[(int64_t)row * g.part_ld + 2 * u.n + half] = make_float2(nan, nan);
        } else if constexpr (kMode == kGrad) {
            const Job& j = g.job[u.job];
            if (j.final && threadIdx.x == 0 && row0 < j.rows && u.n * u.tn < g.d)
                j.to[(int64_t)row0 * j.ld + u.n * u.tn] = 0x7FFF;  // NaN in either type
        }
    }
}

template <bool kPair, int kMode, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1) xent_product_kernel(const __grid_constant__ GemmArgs g)
{
    using S = Shape<kPair, kMode>;
    extern __shared__ uint8_t dyn[];
    __shared__ alignas(8) uint64_t s_full[S::kStages], s_empty[S::kStages], s_acc_full[2], s_acc_empty[2], s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_dead;
    // of the CTAs that share a tile: loads issued, and whether a wait ran out
    __shared__ uint32_t s_steps[2], s_lost[2];

    const int warp = warp_number(), lane = threadIdx.x & 31;
    const uint32_t tiles_at = (smem_addr(dyn) + 1023u) & ~1023u;  // swizzle atoms are 1024 bytes
    const uint32_t rank = kPair ? cluster_rank() : 0;
    const int worker = blockIdx.x / S::kCtas, workers = gridDim.x / S::kCtas;

    let_next_start();
    // what loading and multiplying need first is fetched while the block sets
    // up (1750 clocks between set-up and first load otherwise)
    Tile u, then;
    bool more = false, after = false;
    if (warp >= kResultWarps) {
        more = next_tile(g, worker, workers, 0, u);
        if (warp == kResultWarps && lane < 4 && g.job[lane & 1].tiles > 0)
            prefetch_map(lane < 2 ? &g.a[lane] : &g.b[lane - 2]);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_addr(&s_full[s]), 1);
            mbar_init(smem_addr(&s_empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&s_acc_full[b]), 1);
            mbar_init(smem_addr(&s_acc_empty[b]), kResultWarps * S::kCtas);
        }
        mbar_init(smem_addr(&s_drain), 1);
        s_dead = g.give_up;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 0)
        tmem_alloc<kPair>(smem_addr(&s_tmem), 512);
    fence_before_sync();
    __syncthreads();
    if constexpr (kPair)
        cluster_sync();
    fence_after_sync();
    const uint32_t tmem = s_tmem;
    volatile int* dead = &s_dead;
    if (kMode != kLoss)
        wait_for_previous();
    else if (blockIdx.x == 0 && threadIdx.x == 0)
        g.control->ticket = 0;

    // The loading and the multiplying warp run their loops as whole warps, so
    // that addresses and descriptors stay in uniform registers, and one lane
    // issues; a step has 512 clocks, and every instruction on the way to its
    // four products counts (650 clocks a step with one lane in the loop).
    if (warp == kResultWarps) {
        // ---- loads: this CTA's rows of A and its share of the columns of B
        Ring<S::kStages> ring;
        uint32_t steps = 0;
        const uint32_t stop = g.give_up ? (worker * 2 + rank * 3) % 9 : ~0u;  // either CTA of a pair elsewhere
        bool ok = true;
        const bool one = elect_one();
        for (int k = 1; ok && more; ++k, more = after, u = then) {
            const CUtensorMap* ma = &g.a[u.job];
            const CUtensorMap* mb = &g.b[u.job];
            const int share = u.tn / S::kCtas;
            const int row0 = u.m * S::kTileM + (int)rank * kRows;
            const int col0 = u.n * u.tn + (int)rank * share;
            const uint32_t bytes = (kBytesA + share * (kTileK * 2)) * S::kCtas;
            auto run = [&](auto a_mn, auto b_mn) {
                for (int kb = u.kb0; kb < u.kb1; ++kb, ++steps, ring.next()) {
                    ok = steps != stop && mbar_wait_warp(smem_addr(s_empty) + ring.at * 8, ring.phase ^ 1, dead);
                    if (!ok)
                        break;
                    if (one) {
                        uint32_t full = smem_addr(s_full) + ring.at * 8;
                        const uint32_t at_a = tiles_at + ring.at * S::kStageBytes, at_b = at_a + kBytesA;
                        if (rank == 0)
                            mbar_expect(full, bytes);
                        if constexpr (kPair)
                            full = peer_addr(full, 0);
                        auto load = [&](uint32_t at, const CUtensorMap* m, int x, int y) {
                            if constexpr (kPair)
                                tma_load_pair(at, m, full, x, y);
                            else
                                tma_load(at, m, full, x, y);
                        };
                        if constexpr (a_mn.value) {
#pragma unroll
                            for (int q = 0; q < kRows / 64; ++q)
                                load(at_a + q * kBlock, ma, row0 + q * 64, kb * kTileK);
                        } else {
                            load(at_a, ma, kb * kTileK, row0);
                        }
                        if constexpr (b_mn.value) {
#pragma unroll
                            for (int q = 0; q < kTileN / S::kCtas / 64; ++q)
                                if (q * 64 < share)
                                    load(at_b + q * kBlock, mb, col0 + q * 64, kb * kTileK);
                        } else {
                            load(at_b, mb, kb * kTileK, col0);
                        }
                    }
                    if (kb == u.kb0)  // its divisions run under this tile's loads
                        after = next_tile(g, worker, workers, k, then);
                    __syncwarp();
                }
            };
            by_layout<kMode>(g.job[u.job].is_dw, run);
        }
        // the last products' signals must find this block's barriers
        for (uint32_t b = steps > S::kStages ? steps - S::kStages : 0; ok && b < steps; ++b)
            ok = mbar_wait_warp(smem_addr(s_empty) + (b % S::kStages) * 8, (b / S::kStages) & 1, dead);
        if (lane == 0)
            s_steps[rank] = steps;
    } else if (warp == kResultWarps + 1 && rank == 0) {
        // ---- products
        Ring<S::kStages> ring;
        uint32_t acc = 0;
        bool ok = true;
        const bool one = elect_one();
        for (int k = 1; ok && more; ++k, more = after, u = then) {
            const uint32_t idesc = g.job[u.job].idesc;
            auto run = [&](auto a_mn, auto b_mn) {
                // one product takes 16 of K: 32 bytes along a row, or 16 rows
                constexpr uint32_t step_a = (a_mn.value ? 2048 : 32) >> 4, step_b = (b_mn.value ? 2048 : 32) >> 4;
                const uint64_t desc_a = smem_desc(tiles_at, kBlock, 1024);
                const uint64_t desc_b = smem_desc(tiles_at + kBytesA, kBlock, 1024);
                for (int kb = u.kb0; ok && kb < u.kb1; ++acc) {
                    const uint32_t buf = acc & 1;
                    if (!(ok = mbar_wait_warp(smem_addr(s_acc_empty) + buf * 8, ((acc >> 1) & 1) ^ 1, dead)))
                        break;
                    fence_after_sync();
                    const uint32_t d = tmem + buf * kTileN;
                    const int last = kMode != kGrad ? min(u.kb1 - kb, kPromote) + kb : u.kb1;
                    uint32_t add = 0;
                    // whether the next step's tiles are there is asked before
                    // this step's products are issued
                    bool there = mbar_try(smem_addr(s_full) + ring.at * 8, ring.phase);
                    for (; kb < last; ++kb) {
                        if (!__all_sync(0xffffffffu, there) &&
                            !(ok = mbar_wait_warp(smem_addr(s_full) + ring.at * 8, ring.phase, dead)))
                            break;
                        fence_after_sync();
                        const uint32_t here = ring.at;
                        ring.next();
                        if (kb + 1 < last)
                            there = mbar_try(smem_addr(s_full) + ring.at * 8, ring.phase);
                        const uint64_t a = desc_a + here * (S::kStageBytes >> 4), b = desc_b + here * (S::kStageBytes >> 4);
                        if (one) {
#pragma unroll
                            for (int e = 0; e < kTileK / 16; ++e) {
                                mma_f16<kPair>(d, a + e * step_a, b + e * step_b, idesc, add);
                                add = 1;
                            }
                            mma_commit<kPair>(smem_addr(s_empty) + here * 8);
                        }
                        add = 1;
                        __syncwarp();
                        if (kb == u.kb0)
                            after = next_tile(g, worker, workers, k, then);
                    }
                    if (ok && one)
                        mma_commit<kPair>(smem_addr(s_acc_full) + buf * 8);
                    __syncwarp();
                }
            };
            by_layout<kMode>(g.job[u.job].is_dw, run);
        }
    } else if (warp < kResultWarps) {
        // ---- results
        const int quad = warp & 3;  // a warp reads the 32 lanes of its quarter
        const int half = warp >> 2;
        Box box;
        box.row = quad * 32 + lane;
        box.half = half;
        box.at = tiles_at + S::kStages * S::kStageBytes + half * kOutBytes;
        box.row_at = box.at + box.row * 128;
        box.first = box.row == 0;
        const uint32_t lanes_at = tmem + ((uint32_t)(quad * 32) << 16);
        uint32_t acc = 0;
        bool ok = true;
        auto await = [&]() {
            // one answer in all warps that meet at the barriers of a box
            ok = mbar_wait_warp(smem_addr(&s_acc_full[acc & 1]), (acc >> 1) & 1, dead);
            if constexpr (kMode != kLoss)
                ok = named_all(1 + half, 32 * kResultWarps / 2, ok);
            fence_after_sync();
            return ok;
        };
        auto give_back = [&]() {
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                const uint32_t bar = smem_addr(&s_acc_empty[acc & 1]);
                if constexpr (kPair)
                    mbar_arrive_peer(peer_addr(bar, 0));
                else
                    mbar_arrive(bar);
            }
            ++acc;
        };
        for (int k = 0, t; ok && (t = tile_number(g, worker, workers, k)) >= 0; ++k) {
            const Tile u = tile_at(g, t);
            const int row0 = u.m * S::kTileM + (int)rank * kRows;
            const int width = u.tn / 2, col0 = u.n * u.tn + half * width;
            const Row me = row_at<kMode>(g, row0 + quad * 32 + lane);
            if constexpr (kMode != kGrad) {
                float z[kHalf];
                for (int kb = u.kb0; ok && kb < u.kb1; kb += kPromote) {
                    if (!await())
                        break;
                    const uint32_t at = lanes_at + (acc & 1) * kTileN + half * width;
                    if (kb == u.kb0) {
                        // the first part goes straight to its place; whole
                        // 32 columns are read (what lies beyond is masked)
#pragma unroll
                        for (int c = 0; c < kHalf; c += 32)
                            if (c < width)
                                tmem_load32(at + c, *reinterpret_cast<uint32_t(*)[32]>(z + c));
#pragma unroll
                        for (int c = 0; c < kHalf; c += 32)
                            tmem_wait_load(*reinterpret_cast<uint32_t(*)[32]>(z + c));
                    } else {
#pragma unroll
                        for (int c = 0; c < kHalf; c += 16) {
                            if (c < width) {
                                uint32_t r[16];
                                tmem_load16(at + c, r);
                                tmem_wait_load(r);
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    z[c + k] += __uint_as_float(r[k]);
                            }
                        }
                    }
                    give_back();
                }
                if (ok) {
                    if constexpr (kMode == kLoss)
                        rows_loss(g, 2 * u.n + half, col0, width, row0 + quad * 32 + lane, me, z);
                    else
                        rows_dz<kBf16>(g, col0, width, row0, me, z, box);
                }
            } else {
                if (!await())
                    break;
                const uint32_t at = lanes_at + (acc & 1) * kTileN + half * width;
                if (!g.job[u.job].final)
                    rows_sums(g, g.job[u.job], &g.out[u.job], u.split, col0, width, row0, at, box);
                else
                    rows_final<kBf16>(g, g.job[u.job], &g.out[u.job], col0, width, row0, at, box);
                give_back();
            }
        }
    }
    if (kMode != kLoss && warp < kResultWarps)
        store_wait();
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    bool lost = s_dead != 0;
    if constexpr (kPair) {
        if (threadIdx.x == 0) {  // what either CTA has to know of the other
            s_lost[rank] = lost;
            shared_store_peer(peer_addr(smem_addr(&s_lost[rank]), rank ^ 1), lost);
            shared_store_peer(peer_addr(smem_addr(&s_steps[rank]), rank ^ 1), s_steps[rank]);
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while its pair may still signal it
        lost = (s_lost[0] | s_lost[1]) != 0;
    }
    if (lost) {
        // loads and products in flight end before shared and tensor memory are given up
        if (warp == kResultWarps && rank == 0) {
            drain_loads<kPair, S::kStages>(smem_addr(s_full), s_steps[0], s_steps[kPair ? 1 : 0],
                                           kBytesA + g.job[0].tn / S::kCtas * (kTileK * 2), lane);
        } else if (warp == kResultWarps + 1) {
            if (rank == 0 && elect_one())
                mma_commit<kPair>(smem_addr(&s_drain));
            __syncwarp();
            mbar_wait(smem_addr(&s_drain), 0, nullptr);
        }
        __syncwarp();
        __syncthreads();
        if constexpr (kPair)
            cluster_sync();
    }
    fence_after_sync();
    if (warp == 0)
        tmem_free<kPair>(tmem, 512);
    if (kMode == kLoss && threadIdx.x == 0)
        g.control->status[blockIdx.x] = lost;
    if (lost)
        poison_results<S::kTileM, kMode>(g, worker, workers, rank);
}

// ---------------------------------------------------------------------------
// the forward pass of a few rows
// ---------------------------------------------------------------------------

// One to four rows of hidden: the head is read once and that bounds the pass,
// so every warp streams whole rows of it (four at a time, eight 16-byte loads
// in flight per lane) past the rows of hidden, which stand in shared memory as
// binary32.  One row of 50257 x 1024 takes 18 us (5.8 TB/s), 28 us in the
// product kernel, whose start, two rounds of tiles and last results weigh more
// than its loads; four rows 29 us with the merge, 37 there.
constexpr int kFew = 4;
constexpr int kFewThreads = 256;
constexpr int few_ctas(int64_t rows) { return rows > 2 ? 2 : 3; }  // per SM
constexpr int kFewSmem = 160 * 1024;

// Sums of four values over a warp: lane l gets that of row (l >> 3) & 3.
__device__ __forceinline__ float sum_rows(float a0, float a1, float a2, float a3, int lane)
{
    const bool up = lane & 16, left = lane & 8;
    const float c0 = (up ? a2 : a0) + __shfl_xor_sync(0xffffffffu, up ? a0 : a2, 16);
    const float c1 = (up ? a3 : a1) + __shfl_xor_sync(0xffffffffu, up ? a1 : a3, 16);
    float d = (left ? c1 : c0) + __shfl_xor_sync(0xffffffffu, left ? c0 : c1, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        d += __shfl_xor_sync(0xffffffffu, d, o);
    return d;
}

template <bool kBf16>
__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (kBf16) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
            x[2 * e] = f.x;
            x[2 * e + 1] = f.y;
        }
    }
}

// Adds (m2, s2), a maximum and a sum of exponentials, to (m, s).
__device__ __forceinline__ void add_part(float& m, float& s, float m2, float s2)
{
    const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.0f : top;
    s = s * exp2_fast((m - base) * kLog2e) + s2 * exp2_fast((m2 - base) * kLog2e);
    m = top;
}

template <bool kBf16, int kN>
__global__ void __launch_bounds__(kFewThreads, few_ctas(kN))
xent_few_kernel(const __grid_constant__ GemmArgs g, const uint16_t* hidden, int64_t ld_hidden, const uint16_t* weight,
                int64_t ld_weight)
{
    extern __shared__ float4 s_hidden[];  // [kN][steps][2][32]
    __shared__ float2 s_part[kFewThreads / 32][kN];
    let_next_start();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int steps = (g.d + 255) / 256;
    for (int i = threadIdx.x; i < kN * steps * 32; i += kFewThreads) {
        const int n = i / (steps * 32), k = (i - n * steps * 32) * 8;
        float x[8] = {};
        if (n < g.n && k < g.d)
            widen8<kBf16>(*reinterpret_cast<const uint4*>(hidden + n * ld_hidden + k), x);
        float4* to = s_hidden + (n * steps + k / 256) * 64 + (k & 255) / 8;
        to[0] = make_float4(x[0], x[1], x[2], x[3]);
        to[32] = make_float4(x[4], x[5], x[6], x[7]);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0)
        g.control->ticket = 0;
    int64_t target[kN];
    float m[kN], s[kN];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        target[n] = n < g.n ? target_of(g, n) : -1;
        if (target[n] == g.ignore)
            target[n] = -1;
        m[n] = -INFINITY;
        s[n] = 0.0f;
    }
    __syncthreads();

    const int warps = gridDim.x * (kFewThreads / 32);
    for (int64_t r0 = (int64_t)(blockIdx.x * (kFewThreads / 32) + w) * 4; r0 < g.v; r0 += (int64_t)warps * 4) {
        const uint16_t* row[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            row[q] = weight + min(r0 + q, (int64_t)g.v - 1) * ld_weight + lane * 8;
        float acc[4][kN] = {};
        auto step = [&](const uint4 (&v)[4], int i) {
            float x[4][8];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                widen8<kBf16>(v[q], x[q]);
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                const float4 lo = s_hidden[(n * steps + i) * 64 + lane], hi = s_hidden[(n * steps + i) * 64 + 32 + lane];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    acc[q][n] = fmaf(x[q][0], lo.x, acc[q][n]);
                    acc[q][n] = fmaf(x[q][1], lo.y, acc[q][n]);
                    acc[q][n] = fmaf(x[q][2], lo.z, acc[q][n]);
                    acc[q][n] = fmaf(x[q][3], lo.w, acc[q][n]);
                    acc[q][n] = fmaf(x[q][4], hi.x, acc[q][n]);
                    acc[q][n] = fmaf(x[q][5], hi.y, acc[q][n]);
                    acc[q][n] = fmaf(x[q][6], hi.z, acc[q][n]);
                    acc[q][n] = fmaf(x[q][7], hi.w, acc[q][n]);
                }
            }
        };
        int i = 0;
        for (; (i + 2) * 256 <= g.d; i += 2) {
            uint4 a[4], b[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                a[q] = __ldcs(reinterpret_cast<const uint4*>(row[q] + i * 256));
                b[q] = __ldcs(reinterpret_cast<const uint4*>(row[q] + (i + 1) * 256));
            }
            step(a, i);
            step(b, i + 1);
        }
        for (; i * 256 < g.d; ++i) {
            uint4 a[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                a[q] = i * 256 + lane * 8 < g.d ? __ldcs(reinterpret_cast<const uint4*>(row[q] + i * 256))
                                                : make_uint4(0, 0, 0, 0);
            step(a, i);
        }
        const int64_t u = r0 + ((lane >> 3) & 3);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const float z = sum_rows(acc[0][n], acc[1][n], acc[2][n], acc[3][n], lane);
            if (g.z && n < g.n && u < g.v && (lane & 7) == 0)
                g.z[n * g.z_ld + u] = z;
            if (u < g.v && u != target[n])
                add_part(m[n], s[n], z, 1.0f);
        }
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int o = 8; o <= 16; o <<= 1)
            add_part(m[n], s[n], __shfl_xor_sync(0xffffffffu, m[n], o), __shfl_xor_sync(0xffffffffu, s[n], o));
        if (lane == 0)
            s_part[w][n] = make_float2(m[n], s[n]);
    }
    __syncthreads();
    if (threadIdx.x < kN && threadIdx.x < g.n) {
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kFewThreads / 32; ++k)
            add_part(top, sum, s_part[k][threadIdx.x].x, s_part[k][threadIdx.x].y);
        g.part[(int64_t)threadIdx.x * g.part_ld + blockIdx.x] = make_float2(top, sum);
    }
}

// ---------------------------------------------------------------------------
// row losses, the mean, and dH
// ---------------------------------------------------------------------------

struct MergePart {
    double loss;
    unsigned long long valid;
};

constexpr int kMergeRows = 8;  // rows (warps) per CTA

// The logit of one row's target, d values in binary32 with rounding to
// nearest: a loss is mostly the distance from it.
template <bool kBf16>
__device__ __forceinline__ float target_logit(const uint16_t* h, const uint16_t* w, int d, int lane)
{
    constexpr int kU = 4;  // loads of either row under way
    float s0 = 0.0f, s1 = 0.0f;
    for (int k = lane * 8; k < d; k += kU * 256) {
        uint4 a[kU], b[kU];
#pragma unroll
        for (int e = 0; e < kU; ++e) {
            const bool in = k + e * 256 < d;
            a[e] = in ? __ldg(reinterpret_cast<const uint4*>(h + k + e * 256)) : make_uint4(0, 0, 0, 0);
            b[e] = in ? __ldg(reinterpret_cast<const uint4*>(w + k + e * 256)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < kU; ++e) {
            float x[8], y[8];
            widen8<kBf16>(a[e], x);
            widen8<kBf16>(b[e], y);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                s0 = fmaf(x[i], y[i], s0);
                s1 = fmaf(x[i + 1], y[i + 1], s1);
            }
        }
    }
    float s = s0 + s1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

struct MergeArgs {
    const uint16_t* hidden;
    const uint16_t* weight;
    int64_t ld_hidden, ld_weight;
    float* token_loss;
    float* lse;
    MergePart* parts;      // one per CTA
    int32_t nstatus;
    int32_t mean;
    float scale;
    const float* d_scale;
    float* loss;
    int64_t* n_valid;
};

// The parts of each row (one warp) put together; the CTA that is done last
// adds the rows' losses in a fixed order.
template <bool kBf16>
__global__ void __launch_bounds__(kMergeRows * 32)
xent_merge_kernel(const __grid_constant__ GemmArgs g, const __grid_constant__ MergeArgs a)
{
    __shared__ double s_loss[kMergeRows];
    __shared__ unsigned long long s_valid[kMergeRows];
    __shared__ int s_last, s_bad;
    let_next_start();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int row = blockIdx.x * kMergeRows + w;
    float loss = 0.0f, zt = 0.0f;
    bool valid = false, known = false;
    if (row < g.n) {  // needs the call's inputs only
        const int64_t t = target_of(g, row);
        known = t >= 0 && t < g.v;
        valid = t != g.ignore;
        if (valid && known)
            zt = target_logit<kBf16>(a.hidden + (int64_t)row * a.ld_hidden, a.weight + t * a.ld_weight, g.d, lane);
    }
    wait_for_previous();
    if (row < g.n) {
        // maximum and sum of each lane's parts, then of the lanes'
        const float2* p = g.part + (int64_t)row * g.part_ld;
        float top = -INFINITY, sum = 0.0f;
        constexpr int kU = 16;  // a vocabulary of 50257 in one round
        for (int k = lane; k < g.part_ld; k += 32 * kU) {
            float2 q[kU];
#pragma unroll
            for (int e = 0; e < kU; ++e)
                q[e] = k + 32 * e < g.part_ld ? __ldcg(p + k + 32 * e) : make_float2(-INFINITY, 0.0f);
            float now = top;
#pragma unroll
            for (int e = 0; e < kU; ++e)
                now = fmaxf(now, q[e].x);
            const float base = now == -INFINITY ? 0.0f : now;
            sum *= expf(top - base);
#pragma unroll
            for (int e = 0; e < kU; ++e)
                sum += q[e].y * expf(q[e].x - base);
            top = now;
        }
        float all = top;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
        const float base = all == -INFINITY ? 0.0f : all;
        sum *= expf(top - base);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float others = base + logf(sum);  // -inf where there are none
        float total = others;
        if (valid) {
            if (known) {
                // lse from the larger of the two: with the target far below the
                // others zt + loss would keep the places of zt, and be NaN at -inf
                const float over = others - zt, small = log1pf(expf(-fabsf(over)));
                loss = fmaxf(over, 0.0f) + small;
                total = over > 0.0f ? others + small : zt + loss;
                if (isnan(over) || zt == INFINITY)  // (fmaxf drops a NaN)
                    loss = total = __int_as_float(0x7fc00000);
            } else {
                loss = total = __int_as_float(0x7fc00000);  // no such class
            }
        }
        if (lane == 0) {
            a.token_loss[row] = loss;
            a.lse[row] = total;
        }
    }
    if (lane == 0) {
        s_loss[w] = (double)loss;
        s_valid[w] = valid ? 1 : 0;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        MergePart m{0.0, 0};
        for (int k = 0; k < kMergeRows; ++k) {
            m.loss += s_loss[k];
            m.valid += s_valid[k];
        }
        s_last = 1;
        a.parts[blockIdx.x] = m;
        if (gridDim.x > 1) {
            __threadfence();
            s_last = atomicAdd(&g.control->ticket, 1u) == gridDim.x - 1;
        }
        s_bad = 0;
    }
    __syncthreads();
    if (!s_last)
        return;
    if (gridDim.x > 1)
        __threadfence();
    double sum = 0.0;
    unsigned long long count = 0;
    for (int k = threadIdx.x; k < (int)gridDim.x; k += kMergeRows * 32) {
        sum += __ldcg(&a.parts[k].loss);
        count += __ldcg(&a.parts[k].valid);
    }
    for (int k = threadIdx.x; k < a.nstatus; k += kMergeRows * 32)
        if (g.control->status[k])
            s_bad = 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        count += __shfl_xor_sync(0xffffffffu, count, o);
    }
    if (lane == 0) {
        s_loss[w] = sum;
        s_valid[w] = count;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
        count = 0;
        for (int k = 0; k < kMergeRows; ++k) {
            sum += s_loss[k];
            count += s_valid[k];
        }
        const double by = a.mean && count > 0 ? (double)count : 1.0;
        *a.loss = s_bad ? __int_as_float(0x7fc00000) : (float)(sum / by);
        if (a.n_valid)
            *a.n_valid = (int64_t)count;
        const double S = (double)(a.d_scale ? *a.d_scale : a.scale);
        g.control->gscale = s_bad ? __int_as_float(0x7fc00000) : (float)ldexp(S / by, -(int)g.exponent);
    }
}

// dz from kept logits, as rows_dz makes it: eight columns of four rows to a
// thread, the columns that were multiplied last (and are in L2) first.
constexpr int kDzRows = 4, kDzCols = 8 * 256;

template <bool kBf16>
__global__ void __launch_bounds__(256) xent_dz_kernel(const __grid_constant__ GemmArgs g, uint16_t* dz, int64_t dz_ld)
{
    let_next_start();
    wait_for_previous();
    const int groups = (g.n + kDzRows - 1) / kDzRows, chunks = (g.v + kDzCols - 1) / kDzCols;
    for (int64_t i = blockIdx.x; i < (int64_t)groups * chunks; i += gridDim.x) {
        const int chunk = chunks - 1 - (int)(i / groups), row0 = (int)(i % groups) * kDzRows;
        const int col = chunk * kDzCols + threadIdx.x * 8;
        if (col >= g.v)
            continue;
        float z[kDzRows][8];
        Row me[kDzRows];
#pragma unroll
        for (int q = 0; q < kDzRows; ++q) {
            const int row = min(row0 + q, g.n - 1);
            load32(g.z + (int64_t)row * g.z_ld + col, z[q]);
            me[q] = row_at<kDz>(g, row);
        }
#pragma unroll
        for (int q = 0; q < kDzRows; ++q) {
            if (row0 + q >= g.n)
                break;
            const bool live = me[q].target != g.ignore;
            const float base = fmaf(-me[q].lse, kLog2e, g.exponent);
            const int hit = hit_at(g, me[q].target, col, 8);
            float e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                e[k] = live && col + k < g.v ? exp2_fast(fmaf(z[q][k], kLog2e, base)) : 0.0f;
            if (hit >= 0) {
                const float at_target = ldexpf(expm1f(-me[q].loss), (int)g.exponent);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    e[k] = k == hit ? at_target : e[k];
            }
            *reinterpret_cast<uint4*>(dz + (int64_t)(row0 + q) * dz_ld + col) =
                make_uint4(pack2<kBf16>(e[0], e[1]), pack2<kBf16>(e[2], e[3]), pack2<kBf16>(e[4], e[5]), pack2<kBf16>(e[6], e[7]));
        }
    }
}

// A gradient = T(g * the sum of the splits), eight columns to a thread.
template <bool kBf16>
__global__ void __launch_bounds__(256)
xent_round_kernel(const float* part, int32_t splits, int64_t n, int32_t d, const float* gscale, uint16_t* out,
               int64_t ld, int32_t wide)
{
    wait_for_previous();
    const int32_t per = d / 8;
    const float scale = *gscale;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * per; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int32_t c = (int32_t)(i % per) * 8;
        float x[8] = {};
        for (int s = 0; s < splits; ++s) {
            const float4* p = reinterpret_cast<const float4*>(part + ((int64_t)s * n + row) * d + c);
            const float4 lo = p[0], hi = p[1];
            x[0] += lo.x; x[1] += lo.y; x[2] += lo.z; x[3] += lo.w;
            x[4] += hi.x; x[5] += hi.y; x[6] += hi.z; x[7] += hi.w;
        }
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = pack2<kBf16>(x[2 * e] * scale, x[2 * e + 1] * scale);
        uint16_t* to = out + row * ld + c;
        if (wide) {
            *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                to[2 * e] = (uint16_t)(o[e] & 0xFFFFu);
                to[2 * e + 1] = (uint16_t)(o[e] >> 16);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

struct Plan {
    bool grad = false, want_dh = false, want_dw = false;
    bool dh_final = false;  // one piece, one sum: no sums in between
    bool pair = false;      // two CTAs to a tile
    bool few = false;       // the forward pass of up to kFew rows
    int64_t few_rows = 0, few_smem = 0;
    int64_t tn_loss = 0, tn_dz = 0, tn_grad = 0;  // columns of a tile
    int64_t parts = 0;      // half tiles of the whole vocabulary
    int64_t cut = 0;        // rows that the backward pass takes at a time
    int64_t piece = 0;      // columns of one piece of the backward pass
    int64_t splits = 1;     // of dH's sums over a piece
    int64_t merges = 0;
    bool keep = false;      // the logits
    int64_t z_ld = 0;
    size_t off_z = 0, off_part = 0, off_token = 0, off_lse = 0, off_merge = 0, off_ctl = 0, off_dz = 0,
           off_dh = 0, off_dw = 0, total = 0;
};

// The piece: dz of one piece (of a cut's rows) is at most 256 MB.
constexpr int64_t kPieceBytes = 256ll << 20;
// The longest sum that stays in tensor memory, in blocks of 64.  What the tensor
// cores drop comes to 6.5e-9 of a sum of one sign for each of K: 1.1e-4 of 16384,
// a fifth of binary16's half step.  (dW of 131072 rows in one sum was 8e-4 off,
// of 1048576 rows 7e-3.)  Longer ones are cut, dH's in splits, dW's by its rows,
// and the parts are added with rounding to nearest.
constexpr int64_t kLongestSum = 256;
constexpr int64_t kLeastSplit = 16;  // blocks of 64 in one part of a cut sum

// Columns of a tile: as many as 256, unless narrower tiles, which are a
// multiple of `quantum`, end the last round sooner.  A tile costs its products
// (2 clocks a column and block of K) and some 1500 clocks of its own; wider
// tiles read less, so a narrower one has to gain 3%.  (509 x 50257 x 2048: 240
// columns, 97 -> 94 us; 77 x 1000 x 512: 32 columns, with gradients 35 -> 30 us
// on the device.)
int64_t tile_columns(int64_t mt, int64_t cols, int64_t kb, int64_t workers, int64_t quantum)
{
    int64_t best = 0;
    double least = 0.0;
    for (int64_t tn = kTileN; tn >= std::max<int64_t>(32, quantum); tn -= quantum) {
        const double cost = (double)ceil_div(mt * ceil_div(cols, tn), workers) * (double)(2 * tn * kb + 1500);
        if (best == 0 || cost < 0.97 * least) {
            best = tn;
            least = cost;
        }
    }
    return best;
}

// Whether it is quicker to keep a call's logits in binary32 than to multiply
// them again.  Writing, reading and turning them into dz takes 1.4 ps each
// (through memory); multiplying 2 d operations at 1.4 PFLOP/s, but no less than
// reading the head at 6 TB/s, and 5 us more for a product kernel's start and
// end.  With gradients, on the device: 77 x 1000 x 512 25 us again, 21 kept; 64 x
// 50257 x 1024 122 and 104; 1001 x 50257 x 1024 345 and 338; the same at width
// 512 230 and 243; 8192 x 1000 x 512 85 and 85.
bool keeping_pays(int64_t n, int64_t v, int64_t d)
{
    const double logits = (double)n * (double)v;
    const double again = 5.0 + std::max(logits * 2e-9 * (double)d / 1.4, (double)v * 2e-6 * (double)d / 6.0);
    return logits * 1.4e-6 < again;  // us
}

int make_plan(const mpt_xent_args& a, Plan& p)
{
    p.want_dh = a.grad_hidden != nullptr;
    p.want_dw = a.grad_weight != nullptr;
    p.grad = p.want_dh || p.want_dw;
    p.pair = a.n > kRows;
    const int64_t rows = p.pair ? 2 * kRows : kRows, workers = p.pair ? kMaxCtas / 2 : kMaxCtas;
    p.tn_loss = tile_columns(ceil_div(a.n, rows), a.v, ceil_div(a.d, kTileK), workers, 16);
    p.parts = 2 * ceil_div(a.v, p.tn_loss);
    p.few_rows = a.n <= 1 ? 1 : a.n <= 2 ? 2 : kFew;
    p.few_smem = p.few_rows * round_up(a.d, 256) * 4;
    if (a.n <= kFew && p.few_smem <= kFewSmem) {
        p.few = true;
        p.parts = std::min<int64_t>(ceil_div(a.v, 4 * kFewThreads / 32),
                                    kMaxCtas * std::min<int64_t>(few_ctas(p.few_rows), 220 * 1024 / p.few_smem));
    }
    p.merges = std::max<int64_t>(1, ceil_div(a.n, kMergeRows));
    size_t at = 0;
    auto region = [&](size_t bytes) {
        const size_t here = at;
        at = (size_t)round_up((int64_t)(at + bytes), kAlign);
        return here;
    };
    p.off_ctl = region(sizeof(Control));
    p.off_part = region(sizeof(float2) * (size_t)(a.n * p.parts));
    p.off_token = region(sizeof(float) * (size_t)a.n);
    p.off_lse = region(sizeof(float) * (size_t)a.n);
    p.off_merge = region(sizeof(MergePart) * (size_t)p.merges);
    if (p.grad && a.n > 0) {
        p.cut = round_up(ceil_div(a.n, ceil_div(a.n, kLongestSum * kTileK)), 2 * kRows);
        p.cut = std::min(p.cut, a.n);
        p.piece = std::min(round_up(a.v, kTileN), kPieceBytes / (2 * p.cut) / kTileN * kTileN);
        p.off_dz = region((size_t)(p.cut * p.piece * 2));
        p.z_ld = round_up(ceil_div(a.v, p.tn_loss) * p.tn_loss, 64);
        p.keep = a.n * p.z_ld * 4 <= kPieceBytes && p.piece >= a.v && keeping_pays(a.n, a.v, a.d);
        if (p.keep)
            p.off_z = region((size_t)(a.n * p.z_ld * 4));
        p.tn_dz = tile_columns(ceil_div(p.cut, rows), p.piece, ceil_div(a.d, kTileK), workers, 128);
        // few gradient tiles: narrower ones, so that more CTAs have one
        const int64_t tiles = (p.want_dh ? ceil_div(p.cut, rows) : 0) + (p.want_dw ? ceil_div(p.piece, rows) : 0);
        p.tn_grad = 2 * tiles * ceil_div(a.d, kTileN) <= workers ? 128 : 256;
        if (p.want_dw && p.cut < a.n)
            p.off_dw = region((size_t)(p.piece * a.d * 4));
        if (p.want_dh) {
            // cut dH's sums so that one tile is at most half a CTA's share of the piece's work
            const int64_t kb_v = ceil_div(p.piece, kTileK), kb_n = ceil_div(p.cut, kTileK);
            const int64_t tiles_h = ceil_div(p.cut, kRows) * ceil_div(a.d, kTileN);
            const int64_t tiles_w = p.want_dw ? ceil_div(p.piece, kRows) * ceil_div(a.d, kTileN) : 0;
            const int64_t share = (tiles_h * kb_v + tiles_w * kb_n) / kMaxCtas;
            p.splits = std::min<int64_t>(64, ceil_div(kb_v, std::max<int64_t>(kLeastSplit, share / 2)));
            p.splits = std::max(p.splits, ceil_div(kb_v, kLongestSum));
            p.dh_final = p.splits == 1 && p.piece >= a.v;
            if (!p.dh_final)
                p.off_dh = region((size_t)(p.splits * a.n * a.d * 4));
        }
    }
    p.total = at;
    return MPT_OK;
}

bool args_ok(const mpt_xent_args* a)
{
    if (!a || (a->type != MPT_F16 && a->type != MPT_BF16))
        return false;
    if (a->n < 0 || a->n > (1 << 24) || a->v < 1 || a->v > (1 << 24) || a->d < 8 || a->d > (1 << 20) || a->d % 8 != 0)
        return false;
    if (a->target_bytes != 4 && a->target_bytes != 8)
        return false;
    if (a->reduction != MPT_XENT_MEAN && a->reduction != MPT_XENT_SUM)
        return false;
    // tiles are counted in 31 bits
    if (a->n * a->d >= (int64_t)1 << 38)  // strides of tensor maps have 40 bits
        return false;
    const int64_t most = (int64_t)1 << 30, rows = ceil_div(a->n, kRows), wide = ceil_div(a->d, kTileN);
    return rows * ceil_div(a->v, kTileN) <= most && rows * wide * 64 <= most && ceil_div(a->v, kRows) * wide <= most;
}

// [lo, hi) of rows of d 16-bit values ld apart
struct Span {
    uintptr_t lo, hi;
};
Span rows_span(const void* p, int64_t rows, int64_t ld, int64_t d)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, rows ? lo + (uintptr_t)((rows - 1) * ld + d) * 2 : lo};
}
bool meet(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

bool pointers_ok(const mpt_xent_args& a)
{
    const int64_t big = (int64_t)1 << 39;
    auto rows = [&](const void* p, int64_t ld, uintptr_t align, int64_t quantum) {
        return p && reinterpret_cast<uintptr_t>(p) % align == 0 && ld >= a.d && ld < big && ld % quantum == 0;
    };
    if (!rows(a.weight, a.ld_weight, 16, 8) || !a.loss || (reinterpret_cast<uintptr_t>(a.loss) & 3))
        return false;
    if (a.n > 0 && (!rows(a.hidden, a.ld_hidden, 16, 8) || !a.targets ||
                    reinterpret_cast<uintptr_t>(a.targets) % (uintptr_t)a.target_bytes))
        return false;
    if ((reinterpret_cast<uintptr_t>(a.token_loss) & 3) || (reinterpret_cast<uintptr_t>(a.lse) & 3) ||
        (reinterpret_cast<uintptr_t>(a.n_valid) & 7) || (reinterpret_cast<uintptr_t>(a.d_scale) & 3))
        return false;
    if (a.grad_hidden && !rows(a.grad_hidden, a.ld_grad_hidden, 2, 1))
        return false;
    if (a.grad_weight && !rows(a.grad_weight, a.ld_grad_weight, 2, 1))
        return false;
    // gradients are written while the inputs are still read
    const Span h = rows_span(a.hidden, a.n, a.ld_hidden, a.d), w = rows_span(a.weight, a.v, a.ld_weight, a.d);
    const Span gh = a.grad_hidden ? rows_span(a.grad_hidden, a.n, a.ld_grad_hidden, a.d) : Span{0, 0};
    const Span gw = a.grad_weight ? rows_span(a.grad_weight, a.v, a.ld_grad_weight, a.d) : Span{0, 0};
    return !(meet(h, gh) || meet(h, gw) || meet(w, gh) || meet(w, gw) || meet(gh, gw));
}

using EncodeFn = decltype(&cuTensorMapEncodeTiled);
std::atomic<void*> g_encode{nullptr};

EncodeFn encode_fn()
{
    void* f = g_encode.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        g_encode.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeFn>(f);
}

// [planes], `plane` elements apart, of a row-major matrix, cut into boxes of 128
// bytes by box_rows; what lies outside reads as zero and is not written.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* p, int64_t planes, int64_t plane, int64_t rows,
              int64_t cols, int64_t ld, int box_rows)
{
    EncodeFn f = encode_fn();
    if (!f)
        return false;
    const int64_t width = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)(ld * width), (cuuint64_t)(plane * width)};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / width), (cuuint32_t)box_rows, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return f(m, type, planes ? 3 : 2, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_map(CUtensorMap* m, bool bf16, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows)
{
    return make_map(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p, 0, 0, rows, cols,
                    ld, box_rows);
}

template <class K>
bool allow_smem(K kernel, int bytes)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

template <bool kPair, int kMode, bool kBf16>
bool allow_product()
{
    return allow_smem(xent_product_kernel<kPair, kMode, kBf16>, Shape<kPair, kMode>::kSmem);
}

template <bool kBf16>
bool load_kernels()
{
    cudaFuncAttributes fa;
    return allow_product<false, kLoss, kBf16>() && allow_product<true, kLoss, kBf16>() &&
           allow_product<false, kDz, kBf16>() && allow_product<true, kDz, kBf16>() &&
           allow_product<false, kGrad, kBf16>() && allow_product<true, kGrad, kBf16>() &&
           allow_smem(xent_few_kernel<kBf16, 1>, kFewSmem) && allow_smem(xent_few_kernel<kBf16, 2>, kFewSmem) &&
           allow_smem(xent_few_kernel<kBf16, kFew>, kFewSmem) &&
           cudaFuncGetAttributes(&fa, xent_merge_kernel<kBf16>) == cudaSuccess &&
           cudaFuncGetAttributes(&fa, xent_dz_kernel<kBf16>) == cudaSuccess &&
           cudaFuncGetAttributes(&fa, xent_round_kernel<kBf16>) == cudaSuccess;
}

// Once per device, at its first call: every kernel is loaded and may use its
// shared memory, so that no later call loads code inside a capture.  A failure
// is not remembered.
bool set_up_device()
{
    static std::atomic<uint64_t> done{0};
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return false;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit)
        return true;
    if (!encode_fn() || !load_kernels<false>() || !load_kernels<true>())
        return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

template <bool kBf16, int kN>
cudaError_t launch_few(const GemmArgs& g, const mpt_xent_args& a, const Plan& p, cudaStream_t st)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)p.parts);
    lc.blockDim = dim3(kFewThreads);
    lc.dynamicSmemBytes = (size_t)p.few_smem;
    lc.stream = st;
    return cudaLaunchKernelEx(&lc, xent_few_kernel<kBf16, kN>, g, static_cast<const uint16_t*>(a.hidden), a.ld_hidden,
                              static_cast<const uint16_t*>(a.weight), a.ld_weight);
}

// What mpt_debug_xent_give_up asked of this thread's next call.
thread_local int32_t t_give_up = 0;

template <bool kPair, int kMode, bool kBf16>
cudaError_t launch_shape(GemmArgs& g, cudaStream_t st)
{
    g.give_up = t_give_up >> kMode & 1;
    using S = Shape<kPair, kMode>;
    cudaLaunchConfig_t lc = {};
    const int32_t tiles = g.job[0].tiles + g.job[1].tiles;
    const int32_t workers = std::min(tiles, kMaxCtas / S::kCtas);
    g.late = g.job[0].tiles % workers;
    g.ahead = g.late && g.job[1].tiles
                  ? (int32_t)std::llround((double)g.job[0].kb / g.job[0].splits * g.job[1].splits / g.job[1].kb) : 0;
    lc.gridDim = dim3((unsigned)(workers * S::kCtas));
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = S::kSmem;
    lc.stream = st;
    cudaLaunchAttribute attr[2];
    int attrs = 0;
    if (kPair) {
        attr[attrs].id = cudaLaunchAttributeClusterDimension;
        attr[attrs].val.clusterDim.x = S::kCtas;
        attr[attrs].val.clusterDim.y = 1;
        attr[attrs++].val.clusterDim.z = 1;
    }
    if (kMode != kLoss) {  // the first of the chain follows others' work
        attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[attrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    lc.attrs = attr;
    lc.numAttrs = attrs;
    return cudaLaunchKernelEx(&lc, xent_product_kernel<kPair, kMode, kBf16>, g);
}

template <class K, class... A>
cudaError_t launch_next(K kernel, int64_t grid, int threads, cudaStream_t st, const A&... args)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)grid);
    lc.blockDim = dim3(threads);
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, args...);
}

template <int kMode, bool kBf16>
cudaError_t launch_product(bool pair, GemmArgs& g, cudaStream_t st)
{
    return pair ? launch_shape<true, kMode, kBf16>(g, st) : launch_shape<false, kMode, kBf16>(g, st);
}

void set_job(Job& j, bool pair, bool bf16, int64_t m, int64_t n, int64_t k, int64_t splits, bool a_mn, bool b_mn,
             int64_t band, int64_t tn)
{
    const int rows = pair ? 2 * kRows : kRows;
    j.mt = (int32_t)ceil_div(m, rows);
    j.nt = (int32_t)ceil_div(n, tn);
    j.tn = (int32_t)tn;
    j.kb = (int32_t)ceil_div(k, kTileK);
    j.splits = (int32_t)std::min<int64_t>(splits, j.kb);
    j.band = (int32_t)std::min<int64_t>(band, j.mt);
    j.idesc = mma_desc(bf16, a_mn, b_mn, rows, (int)tn);
    j.tiles = j.mt * j.nt * j.splits;
}

template <bool kBf16>
int enqueue(const mpt_xent_args& a, const Plan& p, char* ws, cudaStream_t st)
{
    Control* control = reinterpret_cast<Control*>(ws + p.off_ctl);
    float* token = a.token_loss ? a.token_loss : reinterpret_cast<float*>(ws + p.off_token);
    float* lse = a.lse ? a.lse : reinterpret_cast<float*>(ws + p.off_lse);
    const bool pair = p.pair;
    // logits: up to 32 MB of hidden stay in L2 while the vocabulary streams by;
    // gradients: one row of tiles reads its part of dz once, and the whole
    // width of the other operand from L2
    const int64_t band = std::max<int64_t>(1, (32ll << 20) / (a.d * 2 * (pair ? 2 * kRows : kRows)));

    GemmArgs g{};
    g.n = (int32_t)a.n;
    g.v = (int32_t)a.v;
    g.d = (int32_t)a.d;
    g.targets = a.targets;
    g.target_bytes = a.target_bytes;
    g.ignore = a.ignore_index;
    g.part = reinterpret_cast<float2*>(ws + p.off_part);
    g.part_ld = (int32_t)p.parts;
    g.control = control;
    g.z = p.keep ? reinterpret_cast<float*>(ws + p.off_z) : nullptr;
    g.z_ld = p.z_ld;
    g.stats = {lse, token};
    g.exponent = kBf16 ? 0.0f : 15.0f;
    g.poison = a.loss;

    MergeArgs m{};
    m.hidden = static_cast<const uint16_t*>(a.hidden);
    m.weight = static_cast<const uint16_t*>(a.weight);
    m.ld_hidden = a.ld_hidden;
    m.ld_weight = a.ld_weight;
    m.token_loss = token;
    m.lse = lse;
    m.parts = reinterpret_cast<MergePart*>(ws + p.off_merge);
    m.mean = a.reduction == MPT_XENT_MEAN;
    m.scale = a.scale;
    m.d_scale = a.d_scale;
    m.loss = a.loss;
    m.n_valid = a.n_valid;

    if (p.few && a.n > 0) {
        const cudaError_t e = p.few_rows == 1   ? launch_few<kBf16, 1>(g, a, p, st)
                              : p.few_rows == 2 ? launch_few<kBf16, 2>(g, a, p, st)
                                                : launch_few<kBf16, kFew>(g, a, p, st);
        if (e != cudaSuccess)
            return MPT_ERR_CUDA;
    } else if (a.n > 0) {
        set_job(g.job[0], pair, kBf16, a.n, a.v, a.d, 1, false, false, band, p.tn_loss);
        if (!make_map(&g.a[0], kBf16, a.hidden, a.n, a.d, a.ld_hidden, kRows) ||
            !make_map(&g.b[0], kBf16, a.weight, a.v, a.d, a.ld_weight, (int)p.tn_loss / (pair ? 2 : 1)))
            return MPT_ERR_CUDA;
        if (launch_product<kLoss, kBf16>(pair, g, st) != cudaSuccess)
            return MPT_ERR_CUDA;
        m.nstatus = pair ? 2 * std::min(g.job[0].tiles, kMaxCtas / 2) : std::min(g.job[0].tiles, kMaxCtas);
    } else if (cudaMemsetAsync(control, 0, sizeof(Control), st) != cudaSuccess) {
        return MPT_ERR_CUDA;
    }
    if (launch_next(xent_merge_kernel<kBf16>, p.merges, kMergeRows * 32, st, g, m) != cudaSuccess)
        return MPT_ERR_CUDA;
    if (!p.grad)
        return MPT_OK;
    if (a.n == 0) {
        if (p.want_dw && cudaMemset2DAsync(a.grad_weight, (size_t)a.ld_grad_weight * 2, 0, (size_t)a.d * 2,
                                           (size_t)a.v, st) != cudaSuccess)
            return MPT_ERR_CUDA;
        return MPT_OK;
    }

    uint16_t* dz = reinterpret_cast<uint16_t*>(ws + p.off_dz);
    auto wide = [](const void* q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld % 8 == 0; };
    float* dh = reinterpret_cast<float*>(ws + p.off_dh);
    float* dw = reinterpret_cast<float*>(ws + p.off_dw);
    // T(gscale * the sum of `parts` planes of rows x d)
    auto round_sums = [&](const float* sums, int32_t parts, int64_t rows, uint16_t* to, int64_t ld) {
        const int64_t blocks = std::min<int64_t>(ceil_div(rows * (a.d / 8), 256), 148 * 8);
        return launch_next(xent_round_kernel<kBf16>, blocks, 256, st, sums, parts, rows, (int32_t)a.d,
                           (const float*)&control->gscale, to, ld, (int32_t)wide(to, ld)) == cudaSuccess;
    };
    const uint16_t* w = static_cast<const uint16_t*>(a.weight);
    uint16_t* grad_w = static_cast<uint16_t*>(a.grad_weight);
    const int32_t splits = p.want_dh ? (int32_t)std::min(p.splits, ceil_div(std::min(p.piece, a.v), kTileK)) : 0;
    const bool dw_final = p.cut >= a.n;
    for (int64_t c0 = 0; c0 < a.v; c0 += p.piece) {
        const int64_t cols = std::min(p.piece, a.v - c0);
        const uint16_t* wp = w + c0 * a.ld_weight;
        for (int64_t r0 = 0; r0 < a.n; r0 += p.cut) {
            const int64_t rows = std::min(p.cut, a.n - r0);
            const uint16_t* hp = m.hidden + r0 * a.ld_hidden;
            GemmArgs z = g;
            z.n = (int32_t)rows;
            z.targets = static_cast<const char*>(a.targets) + r0 * a.target_bytes;
            z.stats = {lse + r0, token + r0};
            z.col0 = (int32_t)c0;
            z.job[0] = z.job[1] = Job{};
            GemmArgs q = z;
            if (p.keep) {  // one piece
                z.z = g.z + r0 * p.z_ld;
                const int64_t items = ceil_div(rows, kDzRows) * ceil_div(a.v, kDzCols);
                if (launch_next(xent_dz_kernel<kBf16>, std::min<int64_t>(items, kMaxCtas * 8), 256, st, z, dz, p.piece) != cudaSuccess)
                    return MPT_ERR_CUDA;
            } else {
                set_job(z.job[0], pair, kBf16, rows, cols, a.d, 1, false, false, band, p.tn_dz);
                if (!make_map(&z.a[0], kBf16, hp, rows, a.d, a.ld_hidden, kRows) ||
                    !make_map(&z.b[0], kBf16, wp, cols, a.d, a.ld_weight, (int)p.tn_dz / (pair ? 2 : 1)) ||
                    !make_map(&z.out[0], kBf16, dz, rows, cols, p.piece, kRows))
                    return MPT_ERR_CUDA;
                if (launch_product<kDz, kBf16>(pair, z, st) != cudaSuccess)
                    return MPT_ERR_CUDA;
            }

            // the job of the longer tiles comes first
            const int64_t kb_h = p.want_dh ? ceil_div(ceil_div(cols, kTileK), splits) : 0;
            const int at_h = kb_h >= ceil_div(rows, kTileK) || !p.want_dw ? 0 : 1, at_w = p.want_dh ? 1 - at_h : 0;
            if (p.want_dh) {
                // (a short last piece may add to the first sums only)
                Job& j = q.job[at_h];
                set_job(j, pair, kBf16, rows, a.d, cols, splits, false, true, 1, p.tn_grad);
                j.add = c0 > 0;
                j.final = p.dh_final;
                j.rows = (int32_t)rows;
                j.to = static_cast<uint16_t*>(a.grad_hidden) + r0 * a.ld_grad_hidden;
                j.ld = a.ld_grad_hidden;
                j.wide = wide(j.to, j.ld);
                if (!make_map(&q.a[at_h], kBf16, dz, rows, cols, p.piece, kRows) ||
                    !make_map(&q.b[at_h], kBf16, wp, cols, a.d, a.ld_weight, kTileK) ||
                    (!j.final && !make_map(&q.out[at_h], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dh + r0 * a.d, splits, a.n * a.d,
                                           rows, a.d, a.d, kRows)) ||
                    (j.final && j.wide && !make_map(&q.out[at_h], kBf16, j.to, rows, a.d, j.ld, kRows)))
                    return MPT_ERR_CUDA;
            }
            if (p.want_dw) {
                Job& j = q.job[at_w];
                set_job(j, pair, kBf16, cols, a.d, rows, 1, true, true, 1, p.tn_grad);
                j.is_dw = 1;
                j.final = dw_final;
                j.add = r0 > 0;
                j.rows = (int32_t)cols;
                j.to = grad_w + c0 * a.ld_grad_weight;
                j.ld = a.ld_grad_weight;
                j.wide = wide(j.to, j.ld);
                if (!make_map(&q.a[at_w], kBf16, dz, rows, cols, p.piece, kTileK) ||
                    !make_map(&q.b[at_w], kBf16, hp, rows, a.d, a.ld_hidden, kTileK) ||
                    (!j.final && !make_map(&q.out[at_w], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dw, 1, cols * a.d, cols, a.d, a.d,
                                           kRows)) ||
                    (j.final && j.wide && !make_map(&q.out[at_w], kBf16, j.to, cols, a.d, j.ld, kRows)))
                    return MPT_ERR_CUDA;
            }
            if (launch_product<kGrad, kBf16>(pair, q, st) != cudaSuccess)
                return MPT_ERR_CUDA;
        }
        if (p.want_dw && !dw_final && !round_sums(dw, 1, cols, grad_w + c0 * a.ld_grad_weight, a.ld_grad_weight))
            return MPT_ERR_CUDA;
    }
    if (p.want_dh && !p.dh_final &&
        !round_sums(dh, splits, a.n, static_cast<uint16_t*>(a.grad_hidden), a.ld_grad_hidden))
        return MPT_ERR_CUDA;
    return MPT_OK;
}

}  // namespace

extern "C" {

int mpt_xent_args_init(mpt_xent_args* args)
{
    if (!args)
        return MPT_ERR_INVALID_ARG;
    std::memset(args, 0, sizeof *args);
    args->type = MPT_F16;
    args->target_bytes = 8;
    args->ignore_index = -100;
    args->reduction = MPT_XENT_MEAN;
    args->scale = 1.0f;
    return MPT_OK;
}

int mpt_debug_xent_give_up(int32_t passes)
{
    if (passes & ~(MPT_XENT_PASS_LOSS | MPT_XENT_PASS_DZ | MPT_XENT_PASS_GRAD))
        return MPT_ERR_INVALID_ARG;
    t_give_up = passes;
    return MPT_OK;
}

int mpt_xent_workspace_bytes(const mpt_xent_args* args, size_t* bytes)
{
    if (!args_ok(args) || !bytes)
        return MPT_ERR_INVALID_ARG;
    Plan p;
    const int rc = make_plan(*args, p);
    if (rc == MPT_OK)
        *bytes = p.total;
    return rc;
}

int mpt_xent(const mpt_xent_args* args, void* d_workspace, size_t ws_bytes, void* cuda_stream)
{
    NvtxRange range("mpt.xent");
    if (!args_ok(args) || !pointers_ok(*args))
        return MPT_ERR_INVALID_ARG;
    if (!args->d_scale && (!std::isfinite(args->scale) || !(args->scale > 0.0f)))
        return MPT_ERR_INVALID_ARG;
    Plan p;
    const int rc = make_plan(*args, p);
    if (rc != MPT_OK)
        return rc;
    if (!d_workspace || reinterpret_cast<uintptr_t>(d_workspace) % kAlign != 0 || ws_bytes < p.total)
        return MPT_ERR_WORKSPACE;
    if (!set_up_device()) {
        cudaGetLastError();
        return MPT_ERR_CUDA;
    }
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    char* ws = static_cast<char*>(d_workspace);
    struct Once {
        ~Once() { t_give_up = 0; }
    } once;
    const int done = args->type == MPT_BF16 ? enqueue<true>(*args, p, ws, st) : enqueue<false>(*args, p, ws, st);
    if (done != MPT_OK)
        cudaGetLastError();  // this call's own error
    return done;
}

}  // extern "C"
