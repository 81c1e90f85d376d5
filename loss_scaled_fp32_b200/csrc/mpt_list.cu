// mpt_list.cu -- global gradient norm over a list of tensors, and clipping
// (mpt_list_* of include/mpt.h).
//
//   s_i  = sum over tensor i of g^2             (binary64)
//   norm = sqrt(sum_i s_i) / S                  coef = clip/norm if clipped
//   out  = T(fp32(g) [* fp32(1/S)] * coef)      each product one rounding
//
// The list is cut once, at creation, into one contiguous share per warp of
// the grid (equal numbers of 512-byte granules, so the shares are balanced
// whatever the tensors' sizes are); what a share holds of one tensor is a
// run.  Both kernels walk the same runs:
//
//   list_norm_kernel   one pass over the gradients: the sum of squares of
//                      every run (no atomics, so the results do not depend
//                      on timing) and one record per CTA
//   list_clip_kernel   adds the CTA records in one fixed order, then scales;
//                      as norm-only finish it writes the result and the
//                      tensors' own norms
//
// Squares are summed in binary64: a product of two binary32 values neither
// overflows nor vanishes there, so no input needs a second, careful pass.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/mpt.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 3;
constexpr int kGranule = 1024;     // bytes: one 32-byte load per lane
constexpr int kPtrSlots = 4;       // pointer tables held on the device at once
constexpr int kLongRuns = 128;
// The clipping pass begins at the ends of the shares.  In the norm pass before
// it the loads of all but this much of the list mark their lines as the first
// to leave L2, so that the ends stay: 355M BF16 values 363 -> 340 us, a ragged
// list of 41M FP32 values 88.6 -> 85.  (Marking the ends as the last to leave
// as well, or the clipping pass's loads as the first, gained less or lost.)
constexpr int64_t kKeepBytes = 64ll << 20;
constexpr size_t kAlign = 256;

// What one warp's share holds of one tensor.
struct __align__(16) Run {
    int64_t begin;   // first element, counted inside the tensor
    int64_t len;     // elements
    int32_t tensor;
    int32_t type;    // MPT_F16, MPT_BF16 or MPT_F32
    int32_t out_type;
    int32_t keep;    // elements at its end that the clipping pass should find in L2
};

// What one CTA adds to the totals.
struct __align__(16) CtaSum {
    double sumsq;
    unsigned long long nonfinite;
};

struct ListArgs {
    const Run* runs;
    const int32_t* warp_runs;       // first run of every warp, and the end
    const int32_t* tensor_runs;     // first run of every tensor, and the end
    const int32_t* long_tensors;    // tensors of more than kLongRuns runs
    const void* const* grads;
    void* const* outs;              // clip only
    double* run_sums;
    CtaSum* cta_sums;
    mpt_check_result* result;
    double* tensor_norms;
    const float* d_scale;           // S on the device, or nullptr
    float scale;                    // S from the host
    float clip;
    int32_t n;
    int32_t n_long;
    int32_t sum_ctas;               // CTAs of the norm pass
    int32_t want_tensor_norms;
    int32_t unscale;
    int32_t identity_skips;         // a factor of 1 leaves nothing to write
};

size_t type_bytes(int32_t t) { return t == MPT_F32 ? 4 : 2; }
bool type_ok(int32_t t) { return t == MPT_F16 || t == MPT_BF16 || t == MPT_F32; }

// ---------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------

template <int kType> struct Elem;
template <> struct Elem<MPT_F16> {
    using T = uint16_t;
    static __device__ __forceinline__ float up(T x) { return __half2float(__ushort_as_half(x)); }
    static __device__ __forceinline__ T down(float x) { return __half_as_ushort(__float2half_rn(x)); }
};
template <> struct Elem<MPT_BF16> {
    using T = uint16_t;
    static __device__ __forceinline__ float up(T x) { return __uint_as_float((uint32_t)x << 16); }
    static __device__ __forceinline__ T down(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
template <> struct Elem<MPT_F32> {
    using T = float;
    static __device__ __forceinline__ float up(T x) { return x; }
    static __device__ __forceinline__ T down(float x) { return x; }
};

// One load or store of a lane: 32 bytes, the memory's own unit.  (Clipping 25M
// FP16 gradients into FP32 took 48 us with 16-byte accesses, 39 with these; the
// norm of 355M FP16 gradients 117 and 113: 6.3 TB/s.)
struct Vec {
    uint32_t w[8];
};
constexpr int kVec = (int)sizeof(Vec);

// kOnce: nothing writes there while the kernel runs.  kHint: `hold` says how
// long L2 is to hold the lines.
template <bool kOnce, bool kHint>
__device__ __forceinline__ Vec load_vec(const void* p, uint64_t hold)
{
    Vec v;
    if constexpr (kHint)
        asm volatile("ld.global.nc.L2::cache_hint.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8], %9;"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                     : "l"(p), "l"(hold));
    else if constexpr (kOnce)
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                     : "l"(p));
    else
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                     : "l"(p)
                     : "memory");
    return v;
}

__device__ __forceinline__ void store_vec(void* p, const uint32_t* w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// The 32 bytes of one load as binary32 values.
template <int kType>
__device__ __forceinline__ void widen(const Vec& v, float* x)
{
    if constexpr (kType == MPT_F32) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = __uint_as_float(v.w[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[2 * k] = Elem<kType>::up((uint16_t)(v.w[k] & 0xFFFFu));
            x[2 * k + 1] = Elem<kType>::up((uint16_t)(v.w[k] >> 16));
        }
    }
}

__device__ __forceinline__ double warp_sum(double x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ---------------------------------------------------------------------------
// the norm pass
// ---------------------------------------------------------------------------

// Sum of squares of one run by one warp.  Four 32-byte loads are in flight
// per lane; elements before the first 32-byte boundary and after the last go
// one to a lane.  kClip: all but the last `keep` elements leave L2 first.
template <int kType, bool kClip>
__device__ __forceinline__ double run_square(const void* base, int64_t begin, int64_t len, int64_t keep, int lane,
                                             uint64_t brief, uint64_t usual)
{
    using T = typename Elem<kType>::T;
    constexpr int kPer = kVec / (int)sizeof(T);
    constexpr int kU = 4;
    const T* g = static_cast<const T*>(base) + begin;
    const int skew = (int)(reinterpret_cast<uintptr_t>(g) & (kVec - 1)) / (int)sizeof(T);
    const int64_t head = min(len, (int64_t)((kPer - skew) % kPer));
    const int64_t nv = (len - head) / kPer;
    const Vec* v = reinterpret_cast<const Vec*>(g + head);
    double a0 = 0.0, a1 = 0.0;
    auto add = [&](const Vec& q) {
        float x[kPer];
        widen<kType>(q, x);
#pragma unroll
        for (int e = 0; e < kPer; e += 2) {
            a0 = fma((double)x[e], (double)x[e], a0);
            a1 = fma((double)x[e + 1], (double)x[e + 1], a1);
        }
    };
    int64_t i = lane;
    const int64_t kept = (len - keep - head) / kPer;  // the first vector that is
    for (; i + (kU - 1) * 32 < nv; i += kU * 32) {
        Vec q[kU];
        const uint64_t hold = i - lane < kept ? brief : usual;
#pragma unroll
        for (int k = 0; k < kU; ++k)
            q[k] = load_vec<true, kClip>(v + i + k * 32, hold);
#pragma unroll
        for (int k = 0; k < kU; ++k)
            add(q[k]);
    }
    if (i - lane < nv) {  // the last, partly filled batch in one round, too
        Vec q[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k) {
            q[k] = Vec{};
            if (i + k * 32 < nv)
                q[k] = load_vec<true, kClip>(v + i + k * 32, i - lane < kept ? brief : usual);
        }
#pragma unroll
        for (int k = 0; k < kU; ++k)
            add(q[k]);
    }
    if (lane < head) {
        const double x = (double)Elem<kType>::up(g[lane]);
        a0 = fma(x, x, a0);
    }
    const int64_t tail = head + nv * kPer;
    if (tail + lane < len) {  // fewer than kPer elements
        const double x = (double)Elem<kType>::up(g[tail + lane]);
        a1 = fma(x, x, a1);
    }
    return warp_sum(a0 + a1);
}

// Non-finite elements of one run (only a run whose sum is not finite).
template <int kType>
__device__ __forceinline__ unsigned long long run_nonfinite(const void* base, int64_t begin, int64_t len,
                                                            int lane)
{
    using T = typename Elem<kType>::T;
    const T* g = static_cast<const T*>(base) + begin;
    unsigned long long c = 0;
    for (int64_t i = lane; i < len; i += 32)
        c += isfinite(Elem<kType>::up(g[i])) ? 0 : 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        c += __shfl_xor_sync(0xffffffffu, c, o);
    return c;
}

template <bool kClip>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) list_norm_kernel(ListArgs a)
{
    __shared__ CtaSum s_warp[kWarps];
    // the finishing kernel may take its place now; it waits for this grid
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int first = a.warp_runs[warp], last = a.warp_runs[warp + 1];
    double total = 0.0;
    unsigned long long bad = 0;
    uint64_t brief = 0, usual = 0;
    if constexpr (kClip) {
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(brief));
        asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(usual));
    }
    for (int r0 = first; r0 < last; r0 += 32) {
        // one lane fetches one run and its tensor's address: the dependent
        // loads of up to 32 runs cost one round trip
        Run mine{};
        const void* base = nullptr;
        if (r0 + lane < last) {
            mine = a.runs[r0 + lane];
            base = a.grads[mine.tensor];
        }
        const int here = min(32, last - r0);
        for (int k = 0; k < here; ++k) {
            const int64_t begin = __shfl_sync(0xffffffffu, mine.begin, k);
            const int64_t len = __shfl_sync(0xffffffffu, mine.len, k);
            const int type = __shfl_sync(0xffffffffu, mine.type, k);
            const void* g = reinterpret_cast<const void*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(base), k));
            const int keep = __shfl_sync(0xffffffffu, mine.keep, k);
            double s = type == MPT_F16    ? run_square<MPT_F16, kClip>(g, begin, len, keep, lane, brief, usual)
                       : type == MPT_BF16 ? run_square<MPT_BF16, kClip>(g, begin, len, keep, lane, brief, usual)
                                          : run_square<MPT_F32, kClip>(g, begin, len, keep, lane, brief, usual);
            if (!isfinite(s)) {
                bad += type == MPT_F16    ? run_nonfinite<MPT_F16>(g, begin, len, lane)
                       : type == MPT_BF16 ? run_nonfinite<MPT_BF16>(g, begin, len, lane)
                                          : run_nonfinite<MPT_F32>(g, begin, len, lane);
                s = __longlong_as_double(0x7ff0000000000000ll);
            }
            if (lane == 0)
                a.run_sums[r0 + k] = s;
            total += s;
        }
    }
    if (lane == 0) {
        s_warp[threadIdx.x >> 5].sumsq = total;
        s_warp[threadIdx.x >> 5].nonfinite = bad;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        CtaSum c{0.0, 0};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            c.sumsq += s_warp[w].sumsq;
            c.nonfinite += s_warp[w].nonfinite;
        }
        a.cta_sums[blockIdx.x] = c;
    }
}

// ---------------------------------------------------------------------------
// the finish and the clipping pass
// ---------------------------------------------------------------------------

struct Totals {
    double norm;
    unsigned long long nonfinite;
    float inv_scale;
    float coef;
    bool clipped;
};

// Every CTA adds the records in the same order: thread t takes t, t + 256, ...
__device__ __forceinline__ Totals totals(const ListArgs& a, CtaSum* s_sum, Totals* s_out)
{
    CtaSum c{0.0, 0};
    for (int k = threadIdx.x; k < a.sum_ctas; k += kThreads) {
        c.sumsq += __ldcg(&a.cta_sums[k].sumsq);
        c.nonfinite += __ldcg(&a.cta_sums[k].nonfinite);
    }
    c.sumsq = warp_sum(c.sumsq);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        c.nonfinite += __shfl_xor_sync(0xffffffffu, c.nonfinite, o);
    if ((threadIdx.x & 31) == 0)
        s_sum[threadIdx.x >> 5] = c;
    __syncthreads();
    if (threadIdx.x == 0) {
        double sum = 0.0;
        unsigned long long bad = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            sum += s_sum[w].sumsq;
            bad += s_sum[w].nonfinite;
        }
        const float S = a.d_scale ? *a.d_scale : a.scale;
        Totals t;
        t.nonfinite = bad;
        t.norm = bad ? __longlong_as_double(0x7ff0000000000000ll) : sqrt(sum) / (double)S;
        t.clipped = !bad && a.clip > 0.0f && t.norm > (double)a.clip;
        t.coef = t.clipped ? __double2float_rn((double)a.clip / t.norm) : 1.0f;
        t.inv_scale = __fdiv_rn(1.0f, S);
        *s_out = t;
    }
    __syncthreads();
    return *s_out;
}

__device__ __forceinline__ void write_result(const ListArgs& a, const Totals& t)
{
    mpt_check_result r;
    r.found_inf = t.nonfinite ? 1 : 0;
    r.clipped = t.clipped ? 1 : 0;
    r.grad_norm = t.norm;
    r.clip_coef = t.coef;
    r.reserved = 0;
    r.n_nonfinite = t.nonfinite;
    *a.result = r;
}

// One warp per tensor, over the whole grid; the few tensors of many runs one
// CTA each (with one warp for the 4096 runs of a million values the norm took
// 18 us, with a CTA 12).
__device__ __forceinline__ void write_tensor_norms(const ListArgs& a)
{
    __shared__ double s_part[kWarps];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const double S = (double)(a.d_scale ? *a.d_scale : a.scale);
    for (int k = blockIdx.x; k < a.n_long; k += gridDim.x) {
        const int i = a.long_tensors[k];
        const int first = a.tensor_runs[i], end = a.tensor_runs[i + 1];
        double s = 0.0;
        for (int r = first + threadIdx.x; r < end; r += 4 * kThreads) {
            double q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q[e] = r + e * kThreads < end ? __ldcg(a.run_sums + r + e * kThreads) : 0.0;
            s += (q[0] + q[1]) + (q[2] + q[3]);
        }
        s = warp_sum(s);
        if (lane == 0)
            s_part[w] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            double t = 0.0;
#pragma unroll
            for (int e = 0; e < kWarps; ++e)
                t += s_part[e];
            a.tensor_norms[i] = sqrt(t) / S;
        }
        __syncthreads();
    }
    for (int i = blockIdx.x * kWarps + w; i < a.n; i += gridDim.x * kWarps) {
        const int first = a.tensor_runs[i], end = a.tensor_runs[i + 1];
        if (end - first > kLongRuns)
            continue;
        double s = 0.0;
        for (int r = first + lane; r < end; r += 32)
            s += __ldcg(a.run_sums + r);
        s = warp_sum(s);
        if (lane == 0)
            a.tensor_norms[i] = sqrt(s) / S;
    }
}

__global__ void __launch_bounds__(kThreads) list_finish_kernel(ListArgs a)
{
    __shared__ CtaSum s_sum[kWarps];
    __shared__ Totals s_tot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0) {
        const Totals t = totals(a, s_sum, &s_tot);
        if (threadIdx.x == 0)
            write_result(a, t);
    }
    if (a.want_tensor_norms)
        write_tensor_norms(a);
}

template <int kIn, int kOut>
__device__ __forceinline__ typename Elem<kOut>::T scaled(float x, float inv, float coef, bool unscale)
{
    if (unscale)
        x = __fmul_rn(x, inv);
    return Elem<kOut>::down(__fmul_rn(x, coef));
}

// One batch of kN 32-byte input vectors, 32 lanes apart, scaled and stored;
// kEnds: those from `end` on are left out.
template <int kIn, int kOut, int kN, bool kEnds>
__device__ __forceinline__ void scale_vecs(const Vec* v, typename Elem<kOut>::T* o, int64_t i, int64_t end,
                                           bool wide, float inv, float coef, bool unscale)
{
    using TO = typename Elem<kOut>::T;
    constexpr int kPer = kVec / (int)sizeof(typename Elem<kIn>::T);
    Vec q[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        q[k] = Vec{};
        if (!kEnds || i + k * 32 < end)
            q[k] = load_vec<false, false>(v + i + k * 32, 0);
    }
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        const bool in = !kEnds || i + k * 32 < end;
        float x[kPer];
        widen<kIn>(q[k], x);
        TO y[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            y[e] = scaled<kIn, kOut>(x[e], inv, coef, unscale);
        TO* to = o + (i + k * 32) * kPer;
        if (in && wide) {
            // kPer outputs are 16, 32 or 64 bytes
            constexpr int kWords = kPer * (int)sizeof(TO) / 4;
            uint32_t w[kWords];
#pragma unroll
            for (int e = 0; e < kWords; ++e) {
                if constexpr (sizeof(TO) == 4)
                    w[e] = __float_as_uint(y[e]);
                else
                    w[e] = (uint32_t)y[2 * e] | ((uint32_t)y[2 * e + 1] << 16);
            }
            if constexpr (kWords == 4) {
                *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int e = 0; e < kWords; e += 8)
                    store_vec(reinterpret_cast<uint32_t*>(to) + e, w + e);
            }
        } else if (in) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                to[e] = y[e];
        }
    }
}

// One run scaled by one warp, from its end to its start: the norm pass left
// the ends of the shares in L2.
template <int kIn, int kOut>
__device__ __forceinline__ void run_scale(const void* base, void* out, int64_t begin, int64_t len,
                                          int lane, float inv, float coef, bool unscale)
{
    using T = typename Elem<kIn>::T;
    using TO = typename Elem<kOut>::T;
    constexpr int kPer = kVec / (int)sizeof(T);
    constexpr int kU = 2;
    const T* g = static_cast<const T*>(base) + begin;
    TO* o = static_cast<TO*>(out) + begin;
    const int skew = (int)(reinterpret_cast<uintptr_t>(g) & (kVec - 1)) / (int)sizeof(T);
    const int64_t head = min(len, (int64_t)((kPer - skew) % kPer));
    const int64_t nv = (len - head) / kPer;
    const int64_t tail = head + nv * kPer;
    const Vec* v = reinterpret_cast<const Vec*>(g + head);
    TO* ov = o + head;
    constexpr int kOutAlign = kPer * (int)sizeof(TO) < kVec ? kPer * (int)sizeof(TO) : kVec;
    const bool wide = (reinterpret_cast<uintptr_t>(ov) & (kOutAlign - 1)) == 0;
    if (tail + lane < len)
        o[tail + lane] = scaled<kIn, kOut>(Elem<kIn>::up(g[tail + lane]), inv, coef, unscale);
    const int64_t full = nv / (kU * 32);
    scale_vecs<kIn, kOut, kU, true>(v, ov, full * (kU * 32) + lane, nv, wide, inv, coef, unscale);
    for (int64_t b = full - 1; b >= 0; --b)
        scale_vecs<kIn, kOut, kU, false>(v, ov, b * (kU * 32) + lane, nv, wide, inv, coef, unscale);
    if (lane < head)
        o[lane] = scaled<kIn, kOut>(Elem<kIn>::up(g[lane]), inv, coef, unscale);
}

template <int kIn>
__device__ __forceinline__ void run_scale_to(int out_type, const void* g, void* o, int64_t begin,
                                             int64_t len, int lane, float inv, float coef, bool unscale)
{
    if (out_type == MPT_F16)
        run_scale<kIn, MPT_F16>(g, o, begin, len, lane, inv, coef, unscale);
    else if (out_type == MPT_BF16)
        run_scale<kIn, MPT_BF16>(g, o, begin, len, lane, inv, coef, unscale);
    else
        run_scale<kIn, MPT_F32>(g, o, begin, len, lane, inv, coef, unscale);
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) list_clip_kernel(ListArgs a)
{
    __shared__ CtaSum s_sum[kWarps];
    __shared__ Totals s_tot;
    const int lane = threadIdx.x & 31;
    const int warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int first = a.warp_runs[warp], last = a.warp_runs[warp + 1];  // written at creation
    // the last 32 runs and their addresses are at hand when the wait ends
    int r0 = first + (last - first - 1) / 32 * 32;
    Run mine{};
    const void* base = nullptr;
    void* to = nullptr;
    auto fetch = [&]() {
        if (r0 + lane < last) {
            mine = a.runs[r0 + lane];
            base = a.grads[mine.tensor];
            to = a.outs[mine.tensor];
        }
    };
    if (first < last)
        fetch();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Totals t = totals(a, s_sum, &s_tot);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        write_result(a, t);
    const bool unscale = a.unscale != 0 && t.inv_scale != 1.0f;
    const bool skip = a.identity_skips && !unscale && t.coef == 1.0f;  // in place, one factor of exactly 1
    while (!skip && first < last) {
        for (int k = min(32, last - r0) - 1; k >= 0; --k) {
            const int64_t begin = __shfl_sync(0xffffffffu, mine.begin, k);
            const int64_t len = __shfl_sync(0xffffffffu, mine.len, k);
            const int type = __shfl_sync(0xffffffffu, mine.type, k);
            const int otype = __shfl_sync(0xffffffffu, mine.out_type, k);
            const void* g = reinterpret_cast<const void*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(base), k));
            void* o = reinterpret_cast<void*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), k));
            if (type == MPT_F16)
                run_scale_to<MPT_F16>(otype, g, o, begin, len, lane, t.inv_scale, t.coef, unscale);
            else if (type == MPT_BF16)
                run_scale_to<MPT_BF16>(otype, g, o, begin, len, lane, t.inv_scale, t.coef, unscale);
            else
                run_scale_to<MPT_F32>(otype, g, o, begin, len, lane, t.inv_scale, t.coef, unscale);
        }
        if (r0 == first)
            break;
        r0 -= 32;
        fetch();
    }
    if (a.want_tensor_norms)
        write_tensor_norms(a);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct Plan {
    std::vector<Run> runs;
    std::vector<int32_t> warp_runs;
    std::vector<int32_t> tensor_runs;
    std::vector<int32_t> long_tensors;
    int32_t ctas = 0;
    size_t off_result = 0, off_norms = 0, off_cta = 0, off_run_sums = 0, off_ptrs = 0, off_runs = 0,
           off_warp = 0, off_tensor = 0, off_long = 0, total = 0;
};

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

constexpr int kMaxCtas = 148 * kCtasPerSm;

int build_plan(const int64_t* sizes, const int32_t* types, const int32_t* out_types, int32_t n, Plan& p)
{
    // granules of the whole list; each tensor costs one more, for its
    // address and its ragged ends
    int64_t units = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (sizes[i] < 0 || !type_ok(types[i]) || (out_types && !type_ok(out_types[i])))
            return MPT_ERR_INVALID_ARG;
        if (sizes[i] > ((int64_t)1 << 48))
            return MPT_ERR_INVALID_ARG;
        if (sizes[i] > 0)
            units += (sizes[i] * (int64_t)type_bytes(types[i]) + kGranule - 1) / kGranule + 1;
        if (units > ((int64_t)1 << 48))  // and units * warps stays in 63 bits
            return MPT_ERR_INVALID_ARG;
    }
    const int64_t warps_max = (int64_t)kMaxCtas * kWarps;
    // at least 2 KB (two loads a lane) to a warp: a million FP16 values are done
    // by 128 CTAs in 8.2 us, by 512 CTAs of a quarter of the work in 10.4 us
    const int64_t warps_wanted = std::max<int64_t>(1, std::min((units + 1) / 2, warps_max));
    p.ctas = (int32_t)((warps_wanted + kWarps - 1) / kWarps);
    const int64_t warps = (int64_t)p.ctas * kWarps;
    p.warp_runs.assign(1, 0);
    p.tensor_runs.assign(1, 0);
    int64_t done = 0;  // granules given out
    int64_t w = 0;     // the warp that takes the next granule
    auto quota_end = [&](int64_t k) { return units * (k + 1) / warps; };
    const int64_t kept = kKeepBytes / kGranule / warps;  // granules at the end of a share
    for (int32_t i = 0; i < n; ++i) {
        const int64_t per = kGranule / (int64_t)type_bytes(types[i]);
        int64_t at = 0;
        if (sizes[i] > 0)
            done += 1;
        while (at < sizes[i]) {
            while (done >= quota_end(w) && w + 1 < warps) {
                p.warp_runs.push_back((int32_t)p.runs.size());
                ++w;
            }
            const int64_t left = (sizes[i] - at + per - 1) / per;
            int64_t take = w + 1 < warps ? std::min(left, quota_end(w) - done) : left;
            Run r{};
            r.begin = at;
            r.len = std::min(sizes[i] - at, take * per);
            r.tensor = i;
            r.type = types[i];
            r.out_type = out_types ? out_types[i] : types[i];
            const int64_t after = quota_end(w) - done - take;  // granules of the share behind this run
            r.keep = (int32_t)std::min(r.len, std::max<int64_t>(0, kept - after) * per);
            p.runs.push_back(r);
            at += r.len;
            done += take;
        }
        if ((int64_t)p.runs.size() - p.tensor_runs.back() > kLongRuns)
            p.long_tensors.push_back(i);
        p.tensor_runs.push_back((int32_t)p.runs.size());
    }
    while ((int64_t)p.warp_runs.size() < warps + 1)
        p.warp_runs.push_back((int32_t)p.runs.size());

    size_t at = 0;
    auto region = [&](size_t bytes) {
        const size_t here = at;
        at = round_up(at + bytes, kAlign);
        return here;
    };
    p.off_result = region(sizeof(mpt_check_result));
    p.off_norms = region(sizeof(double) * (size_t)n);
    p.off_cta = region(sizeof(CtaSum) * (size_t)p.ctas);
    p.off_run_sums = region(sizeof(double) * p.runs.size());
    p.off_ptrs = region(sizeof(void*) * 2 * (size_t)n * kPtrSlots);
    p.off_runs = region(sizeof(Run) * p.runs.size());
    p.off_warp = region(sizeof(int32_t) * p.warp_runs.size());
    p.off_tensor = region(sizeof(int32_t) * p.tensor_runs.size());
    p.off_long = region(sizeof(int32_t) * p.long_tensors.size());
    p.total = at;
    return MPT_OK;
}

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace

struct mpt_list {
    int device = 0;
    int32_t n = 0;
    Plan p;
    std::vector<int64_t> sizes;
    std::vector<int32_t> types, out_types;
    char* ws = nullptr;
    // device copies of the caller's pointer tables (gradients, then outputs)
    struct Slot {
        std::vector<void*> ptrs;
        bool valid = false;
        bool clip = false;      // the table has outputs
        bool in_place = false;  // every output is its gradient, of the same type
        bool captured = false;  // a graph reads it: never rewritten
        uint64_t used = 0;
        void** pinned = nullptr;
        cudaEvent_t copied = nullptr;
    };
    Slot slot[kPtrSlots];
    uint64_t clock = 0;
    int last_slot = 0;
    mpt_check_result* mailbox = nullptr;
    bool broken = false;
};

namespace {

void release(mpt_list* h)
{
    if (!h)
        return;
    // a list may go while this thread captures something else (Python frees one
    // when it likes): nothing here touches a stream
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    const bool relaxed = cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess;
    for (auto& s : h->slot) {
        if (s.copied) {
            if (cudaEventSynchronize(s.copied) != cudaSuccess)  // the copy reads s.pinned
                cudaGetLastError();
            cudaEventDestroy(s.copied);
        }
        if (s.pinned)
            cudaFreeHost(s.pinned);
    }
    if (h->mailbox)
        cudaFreeHost(h->mailbox);
    if (relaxed)
        cudaThreadExchangeStreamCaptureMode(&mode);
    delete h;
}

struct Span {
    uintptr_t lo, hi;
    int32_t tensor;
};

// Outputs may be their own gradients (same address and type) and must
// otherwise touch no gradient and no other output.
bool outputs_ok(const mpt_list* h, void* const* t, bool* in_place)
{
    const int32_t n = h->n;
    std::vector<Span> in, out;
    in.reserve(n);
    out.reserve(n);
    *in_place = true;
    for (int32_t i = 0; i < n; ++i) {
        if (h->sizes[i] == 0)
            continue;
        const uintptr_t g = reinterpret_cast<uintptr_t>(t[i]), o = reinterpret_cast<uintptr_t>(t[n + i]);
        in.push_back({g, g + (size_t)h->sizes[i] * type_bytes(h->types[i]), i});
        out.push_back({o, o + (size_t)h->sizes[i] * type_bytes(h->out_types[i]), i});
        if (g != o || h->types[i] != h->out_types[i])
            *in_place = false;
    }
    auto by_lo = [](const Span& a, const Span& b) { return a.lo < b.lo; };
    std::sort(out.begin(), out.end(), by_lo);
    for (size_t k = 1; k < out.size(); ++k)
        if (out[k].lo < out[k - 1].hi)
            return false;
    // the outputs are disjoint now, so those that meet a gradient are a
    // contiguous stretch of the sorted list; only its own may be there
    for (const Span& s : in) {
        auto it = std::upper_bound(out.begin(), out.end(), s, by_lo);
        if (it != out.begin() && std::prev(it)->hi > s.lo)
            --it;
        for (; it != out.end() && it->lo < s.hi; ++it) {
            const bool own = it->tensor == s.tensor && it->lo == s.lo && it->hi == s.hi &&
                             h->types[s.tensor] == h->out_types[s.tensor];
            if (!own)
                return false;
        }
    }
    return true;
}

int fail_cuda(mpt_list* h)
{
    cudaGetLastError();
    h->broken = true;
    return MPT_ERR_CUDA;
}

// Whether the stream is being captured; false if it cannot be told.
bool is_capturing(cudaStream_t st, bool* capturing)
{
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cap) != cudaSuccess) {
        cudaGetLastError();  // the default stream while another one is captured: nothing was queued
        return false;
    }
    *capturing = cap != cudaStreamCaptureStatusNone;
    return true;
}

// The slot that holds this pointer table on the device.
int find_slot(mpt_list* h, const void* const* grads, void* const* outs, cudaStream_t st, int* out)
{
    const int32_t n = h->n;
    const size_t half = sizeof(void*) * (size_t)n;
    bool capturing = false;
    if (!is_capturing(st, &capturing))
        return MPT_ERR_CUDA;
    // a norm finds its gradients in a clipping's table too; the slot used last
    // is looked at first
    int k = -1;
    for (int j = 0; k < 0 && j < kPtrSlots; ++j) {
        const int i = (h->last_slot + j) % kPtrSlots;
        const auto& s = h->slot[i];
        if (s.valid && (!outs || s.clip) && std::memcmp(s.ptrs.data(), grads, half) == 0 &&
            (!outs || std::memcmp(s.ptrs.data() + n, outs, half) == 0))
            k = i;
    }
    if (k < 0) {
        // (a table that is held has passed these checks)
        for (int32_t i = 0; i < n; ++i) {
            if (h->sizes[i] == 0)
                continue;
            const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]);
            if (g == 0 || g % type_bytes(h->types[i]))
                return MPT_ERR_INVALID_ARG;
            if (outs) {
                const uintptr_t o = reinterpret_cast<uintptr_t>(outs[i]);
                if (o == 0 || o % type_bytes(h->out_types[i]))
                    return MPT_ERR_INVALID_ARG;
            }
        }
        if (capturing)
            return MPT_ERR_INVALID_ARG;  // the copy of a new table must not be recorded
        for (int i = 0; i < kPtrSlots; ++i) {
            const auto& s = h->slot[i];
            if (s.captured)
                continue;
            if (k < 0 || (!s.valid && h->slot[k].valid) ||
                (s.valid == h->slot[k].valid && s.used < h->slot[k].used))
                k = i;
        }
        if (k < 0)
            return MPT_ERR_INVALID_ARG;  // graphs hold every table
        auto& s = h->slot[k];
        std::vector<void*> table(2 * (size_t)n, nullptr);
        std::memcpy(table.data(), grads, half);
        bool in_place = false;
        if (outs) {
            std::memcpy(table.data() + n, outs, half);
            if (!outputs_ok(h, table.data(), &in_place))
                return MPT_ERR_INVALID_ARG;
        }
        if (s.valid && cudaEventSynchronize(s.copied) != cudaSuccess)
            return fail_cuda(h);
        s.valid = false;
        std::memcpy(s.pinned, table.data(), 2 * half);
        void* dst = h->ws + h->p.off_ptrs + (size_t)k * 2 * half;
        if (cudaMemcpyAsync(dst, s.pinned, 2 * half, cudaMemcpyHostToDevice, st) != cudaSuccess ||
            cudaEventRecord(s.copied, st) != cudaSuccess)
            return fail_cuda(h);
        s.ptrs.swap(table);
        s.clip = outs != nullptr;
        s.in_place = in_place;
        s.valid = true;
    }
    h->slot[k].used = ++h->clock;
    h->last_slot = k;
    if (capturing)
        h->slot[k].captured = true;
    *out = k;
    return MPT_OK;
}

template <class K>
cudaError_t launch(K kernel, int grid, bool early, const ListArgs& a, cudaStream_t st)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned int)grid);
    lc.blockDim = dim3(kThreads);
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&lc, kernel, a);
}

int enqueue(mpt_list* h, const void* const* grads, void* const* outs, float scale, const float* d_scale,
            float clip, uint32_t flags, cudaStream_t st)
{
    if (h->broken)
        return MPT_ERR_BROKEN;
    if (flags & ~(MPT_LIST_TENSOR_NORMS | MPT_LIST_UNSCALE))
        return MPT_ERR_INVALID_ARG;
    if (!std::isfinite(clip) || (reinterpret_cast<uintptr_t>(d_scale) & 3) ||
        (!d_scale && (!std::isfinite(scale) || !(scale > 0.0f))))
        return MPT_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return fail_cuda(h);
    if (dev != h->device)
        return MPT_ERR_INVALID_ARG;
    int k = -1;
    const int rc = find_slot(h, grads, outs, st, &k);
    if (rc != MPT_OK)
        return rc;
    const Plan& p = h->p;
    ListArgs a{};
    a.runs = reinterpret_cast<const Run*>(h->ws + p.off_runs);
    a.warp_runs = reinterpret_cast<const int32_t*>(h->ws + p.off_warp);
    a.tensor_runs = reinterpret_cast<const int32_t*>(h->ws + p.off_tensor);
    void** table = reinterpret_cast<void**>(h->ws + p.off_ptrs) + (size_t)k * 2 * h->n;
    a.grads = const_cast<const void* const*>(table);
    a.outs = table + h->n;
    a.run_sums = reinterpret_cast<double*>(h->ws + p.off_run_sums);
    a.cta_sums = reinterpret_cast<CtaSum*>(h->ws + p.off_cta);
    a.result = reinterpret_cast<mpt_check_result*>(h->ws + p.off_result);
    a.tensor_norms = reinterpret_cast<double*>(h->ws + p.off_norms);
    a.d_scale = d_scale;
    a.scale = scale;
    a.clip = clip;
    a.long_tensors = reinterpret_cast<const int32_t*>(h->ws + p.off_long);
    a.n_long = (int32_t)p.long_tensors.size();
    a.n = h->n;
    a.sum_ctas = p.ctas;
    a.want_tensor_norms = (flags & MPT_LIST_TENSOR_NORMS) ? 1 : 0;
    a.unscale = (flags & MPT_LIST_UNSCALE) ? 1 : 0;
    a.identity_skips = outs && h->slot[k].in_place ? 1 : 0;
    cudaError_t e = outs ? launch(list_norm_kernel<true>, p.ctas, false, a, st)
                         : launch(list_norm_kernel<false>, p.ctas, false, a, st);
    if (e != cudaSuccess)
        return fail_cuda(h);
    if (outs) {
        e = launch(list_clip_kernel, p.ctas, true, a, st);
    } else {
        const int grid = a.want_tensor_norms ? std::min(148, std::max((h->n + kWarps - 1) / kWarps, a.n_long)) : 1;
        e = launch(list_finish_kernel, grid, true, a, st);
    }
    return e == cudaSuccess ? MPT_OK : fail_cuda(h);
}

}  // namespace

extern "C" {

int mpt_list_workspace_bytes(const int64_t* sizes, const int32_t* types, const int32_t* out_types,
                             int32_t n, size_t* bytes)
{
    if (!sizes || !types || n <= 0 || !bytes)
        return MPT_ERR_INVALID_ARG;
    try {
        Plan p;
        const int rc = build_plan(sizes, types, out_types, n, p);
        if (rc == MPT_OK)
            *bytes = p.total;
        return rc;
    } catch (...) {
        return MPT_ERR_INVALID_ARG;
    }
}

int mpt_list_create(const int64_t* sizes, const int32_t* types, const int32_t* out_types, int32_t n,
                    void* d_workspace, size_t ws_bytes, mpt_list** out)
{
    if (!sizes || !types || n <= 0 || !out)
        return MPT_ERR_INVALID_ARG;
    *out = nullptr;
    mpt_list* h = new (std::nothrow) mpt_list();
    if (!h)
        return MPT_ERR_INVALID_ARG;
    int rc = MPT_ERR_INVALID_ARG;
    try {
        rc = build_plan(sizes, types, out_types, n, h->p);
        if (rc == MPT_OK) {
            h->sizes.assign(sizes, sizes + n);
            h->types.assign(types, types + n);
            h->out_types.assign(out_types ? out_types : types, (out_types ? out_types : types) + n);
        }
    } catch (...) {
        rc = MPT_ERR_INVALID_ARG;
    }
    if (rc != MPT_OK) {
        release(h);
        return rc;
    }
    h->n = n;
    const Plan& p = h->p;
    if (!d_workspace || reinterpret_cast<uintptr_t>(d_workspace) % kAlign != 0 || ws_bytes < p.total) {
        release(h);
        return MPT_ERR_WORKSPACE;
    }
    if (cudaGetDevice(&h->device) != cudaSuccess) {
        cudaGetLastError();
        release(h);
        return MPT_ERR_CUDA;
    }
    cudaPointerAttributes attr;
    if (cudaPointerGetAttributes(&attr, d_workspace) != cudaSuccess ||
        attr.type != cudaMemoryTypeDevice || attr.device != h->device) {
        cudaGetLastError();
        release(h);
        return MPT_ERR_WORKSPACE;
    }
    char* ws = static_cast<char*>(d_workspace);
    h->ws = ws;
    auto upload = [](void* to, const void* from, size_t bytes) {
        return bytes == 0 || cudaMemcpy(to, from, bytes, cudaMemcpyHostToDevice) == cudaSuccess;
    };
    cudaFuncAttributes fa;  // loads the kernels, so that no later call loads code inside a capture
    // the workspace may come from a stream that still writes what was there before
    bool ok = cudaDeviceSynchronize() == cudaSuccess &&
              cudaFuncGetAttributes(&fa, list_norm_kernel<false>) == cudaSuccess &&
              cudaFuncGetAttributes(&fa, list_norm_kernel<true>) == cudaSuccess &&
              cudaFuncGetAttributes(&fa, list_clip_kernel) == cudaSuccess &&
              cudaFuncGetAttributes(&fa, list_finish_kernel) == cudaSuccess &&
              upload(ws + p.off_runs, p.runs.data(), sizeof(Run) * p.runs.size()) &&
              upload(ws + p.off_warp, p.warp_runs.data(), sizeof(int32_t) * p.warp_runs.size()) &&
              upload(ws + p.off_tensor, p.tensor_runs.data(), sizeof(int32_t) * p.tensor_runs.size()) &&
              upload(ws + p.off_long, p.long_tensors.data(), sizeof(int32_t) * p.long_tensors.size()) &&
              cudaMemset(ws, 0, p.off_ptrs) == cudaSuccess &&
              cudaHostAlloc(reinterpret_cast<void**>(&h->mailbox), sizeof(mpt_check_result), cudaHostAllocDefault) == cudaSuccess;
    for (auto& s : h->slot)
        ok = ok && cudaHostAlloc(reinterpret_cast<void**>(&s.pinned), sizeof(void*) * 2 * (size_t)n, cudaHostAllocDefault) == cudaSuccess &&
             cudaEventCreateWithFlags(&s.copied, cudaEventDisableTiming) == cudaSuccess;
    ok = ok && cudaDeviceSynchronize() == cudaSuccess;
    if (!ok) {
        cudaGetLastError();
        release(h);
        return MPT_ERR_CUDA;
    }
    *out = h;
    return MPT_OK;
}

int mpt_list_norm(mpt_list* h, const void* const* d_grads, float scale, const float* d_scale, float clip,
                  uint32_t flags, void* cuda_stream)
{
    NvtxRange range("mpt.list_norm");
    if (!h || !d_grads || (flags & MPT_LIST_UNSCALE))
        return MPT_ERR_INVALID_ARG;
    try {
        return enqueue(h, d_grads, nullptr, scale, d_scale, clip, flags, static_cast<cudaStream_t>(cuda_stream));
    } catch (...) {
        return MPT_ERR_INVALID_ARG;
    }
}

int mpt_list_clip(mpt_list* h, const void* const* d_grads, void* const* d_out, float scale,
                  const float* d_scale, float clip, uint32_t flags, void* cuda_stream)
{
    NvtxRange range("mpt.list_clip");
    if (!h || !d_grads || !d_out)
        return MPT_ERR_INVALID_ARG;
    try {
        return enqueue(h, d_grads, d_out, scale, d_scale, clip, flags, static_cast<cudaStream_t>(cuda_stream));
    } catch (...) {
        return MPT_ERR_INVALID_ARG;
    }
}

int mpt_list_views(const mpt_list* h, mpt_check_result** d_result, double** d_tensor_norms)
{
    if (!h)
        return MPT_ERR_INVALID_ARG;
    if (d_result)
        *d_result = reinterpret_cast<mpt_check_result*>(h->ws + h->p.off_result);
    if (d_tensor_norms)
        *d_tensor_norms = reinterpret_cast<double*>(h->ws + h->p.off_norms);
    return MPT_OK;
}

int mpt_list_wait(mpt_list* h, void* cuda_stream, mpt_check_result* out)
{
    NvtxRange range("mpt.list_wait");
    if (!h)
        return MPT_ERR_INVALID_ARG;
    if (h->broken)
        return MPT_ERR_BROKEN;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return fail_cuda(h);
    if (dev != h->device)  // whose default stream would be waited for
        return MPT_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    bool capturing = false;
    if (!is_capturing(st, &capturing))
        return MPT_ERR_CUDA;
    if (capturing)
        return MPT_ERR_INVALID_ARG;  // nothing runs that could be waited for
    if (cudaMemcpyAsync(h->mailbox, h->ws + h->p.off_result, sizeof(mpt_check_result),
                        cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return fail_cuda(h);
    if (out)
        *out = *h->mailbox;
    return MPT_OK;
}

int mpt_list_destroy(mpt_list* h)
{
    release(h);
    return MPT_OK;
}

}  // extern "C"
