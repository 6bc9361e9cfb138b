// beam_kernels.cuh -- beam search over the LM head's logits: the best
// continuations over beams and vocabulary, and the beams' states put in the
// order of their parents.
//
// Selection.  A continuation of beam w by token v scores
//     total(w, v) = score_w + x_wv - lse_w,   lse_w = log sum_v exp(x_wv).
// Within a row the order is that of the logits, so the best C of a row are
// among the best C logits of each of its parts, and one pass over the logits
// gives both those and the part's share of lse_w:
//   beam_scan_kernel   one CTA per part of a row: sum of exponentials, best C
//                      logits.  A stream like the cross-entropy forward that also
//                      notes the maximum of each thread's 16 logits; the maxima
//                      give a threshold that C logits reach and few others, and
//                      only the sixteens that reach it are looked at again (66 us at
//                      512 x 151936, 4.9 TB/s; candidates kept as they stream, against
//                      the threshold of the first batch, cost 33 instructions per
//                      logit and 103 us)
//   beam_merge_kernel  one CTA per batch entry: lse of every beam, the best C
//                      of all beams' candidates, the beams that go on
// Continuations are compared by the FP64 value of total, ties by the lower beam, then
// the higher logit (where FP64 cannot tell totals apart that differ), then the lower
// token: an FP32 total has a step of 1e-6 at -15, which the gaps between
// candidates of a large batch do meet.  Within a beam the order is exact; between
// beams it is as good as lse (see beam_scan_kernel).
#pragma once
#include <cfloat>
#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace lmh {

constexpr int kBeamThreads = 256;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamPerThread = 16;                         // logits of a batch, per thread
constexpr int kBeamBatch = kBeamThreads * kBeamPerThread;  // logits of a batch
constexpr int kBeamMaxBatches = 8;                        // batches of a part, at most
constexpr int kBeamBuf = 512;        // candidates at or above the threshold a CTA can hold
constexpr int kBeamHits = 128;        // sixteens at or above it that a warp can list
constexpr int kBeamMaxCand = 128;
constexpr int kBeamMaxWidth = 64;
constexpr float kBeamMaxLogit = 1e38f;
// A reference beyond this (a largest logit beyond about 2^29 either way, as where a
// mask of the type's lowest value covers a part) is too coarse an FP32 number to
// stand in for the largest logit.
constexpr float kBeamMaxRef = 7.7e8f;
constexpr int kBeamDevBadLogit = 0x4;   // LMH_DEV_BAD_LOGIT
constexpr int kBeamDevBadParent = 0x10; // LMH_DEV_BAD_PARENT

// A part's share of its row.
struct BeamPartial {
    double sum;     // sum of 2^(x log2(e) - ref)
    float ref;      // beam_ref(largest logit); -inf if no finite logit;
                    // FLT_MAX, -FLT_MAX beyond kBeamMaxRef: then sum of exp(x - max)
    int32_t count;  // candidates in the part's list
};

struct BeamCand {
    float x;      // the logit
    int32_t tok;  // its token
};

// Order-preserving map of a float to an unsigned integer (-inf lowest).
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float from_ordered(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

constexpr float kLog2e = 1.44269502162933349609f, kLog2eRest = 1.92596303e-8f;  // together log2(e)
constexpr double kLog2eF64 = 1.4426950408889634074;

// The integer power of two that sums are held against whose largest logit is x.
__device__ __forceinline__ float beam_ref(float x) { return fmaxf(rintf(x * kLog2e), -FLT_MAX); }

// 2^d for a whole number d <= 0 (0 below 2^-1022).
__device__ __forceinline__ double pow2(float d)
{
    return d < -1022.f ? 0.0 : __hiloint2double((static_cast<int>(d) + 1023) << 20, 0);
}

// How many of n keys are ahead of a candidate, counted by eight neighbouring lanes
// (`part` is the lane's place among them); every lane gets the result.
template <typename F>
__device__ __forceinline__ int beam_rank(int part, int n, F is_ahead)
{
    int rank = 0;
    for (int j = part; j < n; j += 8)
        rank += is_ahead(j);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
        rank += __shfl_xor_sync(0xffffffffu, rank, o);
    return rank;
}

// A value that at least `want` of the block's per-thread maxima reach, found
// from the q-th largest maximum of each warp: the h-th largest of those, with
// h warps x q lanes >= want.  Of 8 warps, h = 4 lets about twice `want` values
// through for a small `want` (h = 1 about six times as many, h = 8 three times);
// from 32 on all 8 do, since the last few of a warp's 32 maxima are low.  -inf
// when too few threads hold a finite value.  `red` has kBeamWarps entries.
__device__ __forceinline__ float block_threshold(float best, int want, uint32_t *red)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = want >= 32 ? 8 : 4;
    const int q = (want + h - 1) / h;
    uint32_t key = ordered(best), kth = 0;
    for (int i = 0; i < q; ++i) {
        kth = __reduce_max_sync(0xffffffffu, key);
        const unsigned at = __ballot_sync(0xffffffffu, key == kth);
        if (lane == __ffs(at) - 1)
            key = 0;
    }
    if (lane == 0)
        red[warp] = kth;
    __syncthreads();
    key = lane < kBeamWarps ? red[lane] : 0;
    for (int i = 0; i < h; ++i) {
        kth = __reduce_max_sync(0xffffffffu, key);
        const unsigned at = __ballot_sync(0xffffffffu, key == kth);
        if (lane == __ffs(at) - 1)
            key = 0;
    }
    return from_ordered(kth);
}

__device__ __forceinline__ uint4 ldg_vec(const void *p)
{
    uint4 u;
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    return u;
}

template <typename T>
struct BeamVec;
template <>
struct BeamVec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint32_t (&u)[4], float *x)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = __uint_as_float(u[i]);
    }
    static __device__ __forceinline__ float one(const float *p) { return *p; }
};
template <>
struct BeamVec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint32_t (&u)[4], float *x)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ float one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
};

// The 16 bytes that begin `bytes` (0 <= bytes < 16, a multiple of 2) past the
// 16-byte boundary p, out of the vectors they lie in (one where bytes is 0).
__device__ __forceinline__ void ldg_straddle(const void *p, int bytes, uint32_t (&u)[4])
{
    const uint4 a = ldg_vec(p);
    uint4 b = a;
    if (bytes)
        b = ldg_vec(static_cast<const uint4 *>(p) + 1);
    uint32_t w[5];  // the words from the one that holds the first byte on
    switch (bytes >> 2) {
    case 0: w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x; break;
    case 1: w[0] = a.y, w[1] = a.z, w[2] = a.w, w[3] = b.x, w[4] = b.y; break;
    case 2: w[0] = a.z, w[1] = a.w, w[2] = b.x, w[3] = b.y, w[4] = b.z; break;
    default: w[0] = a.w, w[1] = b.x, w[2] = b.y, w[3] = b.z, w[4] = b.w; break;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = __funnelshift_r(w[i], w[i + 1], (bytes & 2) * 8);
}

__device__ __forceinline__ bool beam_live(float score) { return score > -INFINITY && score < INFINITY; }

// Logits [v0, v0 + kBeamBatch) of a row into registers, -inf past the row's end.
// A logit's thread and place go by its column alone, so that equal rows give equal
// sums and their ties fall by beam number wherever the rows start (V may be odd).
// A row that does not start on 16 bytes is read in the aligned vectors around each
// 16 bytes (the second of the two is the neighbour's first, an L1 hit), and its
// first and last elements one by one.
template <typename T>
__device__ __forceinline__ void beam_load(const T *x0, int64_t v0, int64_t V, int off, float (&x)[kBeamPerThread])
{
    constexpr int VN = BeamVec<T>::N;
    const int tid = threadIdx.x;
    if (off == 0 && v0 + kBeamBatch <= V) {  // every load in flight at once
        const uint4 *p = reinterpret_cast<const uint4 *>(x0 + v0) + tid;
        uint4 q[kBeamPerThread / VN];
#pragma unroll
        for (int i = 0; i < kBeamPerThread / VN; ++i)
            q[i] = ldg_vec(p + i * kBeamThreads);
#pragma unroll
        for (int i = 0; i < kBeamPerThread / VN; ++i) {
            const uint32_t u[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
            BeamVec<T>::unpack(u, x + i * VN);
        }
        return;
    }
    const int offe = off / static_cast<int>(sizeof(T));
#pragma unroll
    for (int i = 0; i < kBeamPerThread / VN; ++i) {
        const int64_t v = v0 + (i * kBeamThreads + tid) * VN;
        if (v >= offe && v - offe + (off ? 2 : 1) * VN <= V) {
            uint32_t u[4];
            ldg_straddle(x0 + v - offe, off, u);
            BeamVec<T>::unpack(u, x + i * VN);
        } else {
#pragma unroll
            for (int e = 0; e < VN; ++e)
                x[i * VN + e] = v + e < V ? BeamVec<T>::one(x0 + v + e) : -INFINITY;
        }
    }
}

// Token of element i of thread tid's batch that starts at v0.
template <typename T>
__device__ __forceinline__ int64_t beam_token(int64_t v0, int i, int tid)
{
    constexpr int VN = BeamVec<T>::N;
    return v0 + ((i / VN) * kBeamThreads + tid) * VN + i % VN;
}

// Higher is better: the logit first (-0 as 0), then the lower token.
__device__ __forceinline__ uint64_t beam_key(float x, int64_t tok)
{
    return (static_cast<uint64_t>(ordered(x + 0.f)) << 32) | (0xffffffffu - static_cast<uint32_t>(tok));
}

// Makes unusable logits -inf; whether there were any.
__device__ __forceinline__ bool beam_clean(float (&x)[kBeamPerThread])
{
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kBeamPerThread; ++i) {
        const bool ok = x[i] < kBeamMaxLogit;  // NaN, +inf and what log2(e) times would be: -inf
        bad |= !ok;
        x[i] = ok ? x[i] : -INFINITY;
    }
    return bad;
}

// The sum of a part whose largest logit is beyond kBeamMaxRef's: again, against that
// logit, the first of its list.  All threads of the part's CTA; a call, and all it
// needs made anew, so that the scan has its registers to itself (in line: 512 x 151936
// takes 3 % longer).
template <typename T>
__device__ __noinline__ void beam_sum_far(const T *logits, const BeamCand *cand, BeamPartial *part, int64_t V,
                                          int32_t C, int32_t parts, int32_t batches, double *red_sum)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x / static_cast<unsigned>(parts);
    const T *x0 = logits + row * V;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x0) & 15);
    const int64_t begin = (static_cast<int64_t>(blockIdx.x) - row * parts) * batches * kBeamBatch;
    __syncthreads();  // the list is written, the first sums are read
    const float m = *const_cast<const volatile float *>(&cand[static_cast<int64_t>(blockIdx.x) * C].x);
    double s = 0.0;
    for (int b = 0; b < batches && begin + b * kBeamBatch < V; ++b) {
        float x[kBeamPerThread];
        beam_load(x0, begin + b * kBeamBatch, V, off, x);
        beam_clean(x);
#pragma unroll
        for (int i = 0; i < kBeamPerThread; ++i)
            s += static_cast<double>(expf(x[i] - m));
    }
    s = warp_sum(s);
    if (lane == 0)
        red_sum[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kBeamWarps; ++i)
            s += red_sum[i];
        part[blockIdx.x].sum = s;
        part[blockIdx.x].ref = copysignf(FLT_MAX, m);
    }
}

// One CTA per part (`batches` batches) of a row.  Rows of beams that cannot go on
// (score -inf) and of entries that are done are not read.
template <typename T>
__global__ void __launch_bounds__(kBeamThreads, 6)
    beam_scan_kernel(const T *__restrict__ logits, const float *__restrict__ scores,
                     const int32_t *__restrict__ done, BeamPartial *__restrict__ part,
                     BeamCand *__restrict__ cand, int32_t W, int64_t V, int32_t C, int32_t parts,
                     int32_t batches, int32_t *status)
{
    __shared__ uint32_t red[kBeamWarps];
    __shared__ float red_top[kBeamWarps];
    __shared__ double red_sum[kBeamWarps];
    // of each thread's batch: its maximum, and its sum against beam_ref(maximum)
    __shared__ float2 noted[kBeamMaxBatches][kBeamThreads];
    __shared__ uint16_t listed[kBeamWarps][kBeamHits];  // batch << 5 | lane
    __shared__ uint64_t buf[kBeamBuf];
    __shared__ uint64_t win[kBeamWarps];
    __shared__ int count;
    pdl_wait();
    pdl_launch_dependents();
    const unsigned row32 = blockIdx.x / static_cast<unsigned>(parts);
    const int64_t row = row32;
    const int pt = static_cast<int>(blockIdx.x - row32 * parts);
    if ((done && done[row32 / static_cast<unsigned>(W)]) || !beam_live(scores[row]))
        return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T *x0 = logits + row * V;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x0) & 15);  // bytes past a boundary
    const int64_t begin = static_cast<int64_t>(pt) * batches * kBeamBatch;
    const int64_t end = begin + static_cast<int64_t>(batches) * kBeamBatch < V
                            ? begin + static_cast<int64_t>(batches) * kBeamBatch : V;
    if (tid == 0)
        count = 0;

    // Sums of exponentials against an integer power of two 2^ref: x log2(e) - ref is
    // rounded once per term, near its own size (log2(e) as two floats, so that
    // large logits keep their last places), and sums of different refs are joined by
    // exact scaling.  Each sixteen has the ref of its own largest logit, so that the
    // terms that count have small exponents.  A term is off by up to 2^-20 of itself
    // (ex2.approx 2^-22, the argument's roundings, FP32 sums of 16), which is too much
    // for a row that one token dominates: 5e-7 of lse, more than what separates close
    // beams.  The sixteens looked at again below, which hold the part's best C logits,
    // are therefore summed in FP64 there, and lse is off by at most 2^-20 of the share
    // the others hold (for logits up to 1e7).  Measured with 40 likely tokens:
    // 1e-9 with 16 candidates, 1.8e-8 with one (6e-8 with ex2.approx alone); with a bulk
    // of many terms 3.6e-8, nearly the same for every row.  512 x 151936, selection and
    // merge: 69 us against 66.
    float most = -INFINITY;
    bool any_bad = false;
    int nb = 0;
    for (int64_t v0 = begin; v0 < end; v0 += kBeamBatch, ++nb) {
        float x[kBeamPerThread];
        beam_load(x0, v0, V, off, x);
        float best;
        auto add = [&]() -> float {
            const float ref = beam_ref(best);
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kBeamPerThread; ++i) {
                const float t = fmaf(x[i], kLog2eRest, fmaf(x[i], kLog2e, -ref));
                float y;
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
                s4[i & 3] += y;
            }
            return (s4[0] + s4[1]) + (s4[2] + s4[3]);
        };
        // A NaN or an infinity shows in the sum (fmaxf passes over NaN): once more then.
        float s;
        bool again = false;
        do {
            if (again)
                any_bad |= beam_clean(x);
            best = x[0];
#pragma unroll
            for (int i = 1; i < kBeamPerThread; ++i)
                best = fmaxf(best, x[i]);
            s = best < kBeamMaxLogit ? add() : NAN;
            if (again && !(s < INFINITY))
                s = 0.f;  // logits beyond kBeamMaxRef's: see beam_sum_far
            again = !again && !(s < INFINITY);
        } while (again);
        noted[nb][tid] = make_float2(best, s);
        most = fmaxf(most, best);
    }
    const float warp_top = from_ordered(__reduce_max_sync(0xffffffffu, ordered(most)));
    if (lane == 0)
        red_top[warp] = warp_top;
    const float thr = block_threshold(most, C, red);
    float top = red_top[0];
#pragma unroll
    for (int i = 1; i < kBeamWarps; ++i)
        top = fmaxf(top, red_top[i]);
    const float ref = top > -INFINITY ? beam_ref(top) : -INFINITY;
    double sum = 0.0;
    // The sixteens that reach it: listed by the warp, then two at a time, a lane per
    // logit (the loads are what takes time here).  The others' sums are joined.
    static_assert(kBeamPerThread == 16, "half a warp reads one thread's batch");
    int hits = 0;
    for (int b = 0; b < nb; ++b) {
        const float2 mine = noted[b][tid];
        const bool hit = mine.x >= thr && mine.x > -INFINITY;
        if (!hit && mine.x > -INFINITY)
            sum += static_cast<double>(mine.y) * pow2(beam_ref(mine.x) - ref);
        const unsigned all = __ballot_sync(0xffffffffu, hit);
        const int place = hits + __popc(all & ((1u << lane) - 1u));
        if (hit && place < kBeamHits)
            listed[warp][place] = static_cast<uint16_t>(b << 5 | lane);
        hits += __popc(all);
    }
    __syncwarp();
    if (hits > kBeamHits) {
        hits = 0;
        if (lane == 0)
            atomicAdd(&count, kBeamBuf + 1);  // as when the buffer is full
    }
    for (int i = 0; i < hits; i += 2) {
        const int mine = i + (lane >> 4);
        const int at_hit = mine < hits ? listed[warp][mine] : 0;
        const int64_t v = beam_token<T>(begin + static_cast<int64_t>(at_hit >> 5) * kBeamBatch, lane & 15,
                                        warp * 32 + (at_hit & 31));
        float x = mine < hits && v < V ? BeamVec<T>::one(x0 + v) : -INFINITY;
        x = x < kBeamMaxLogit ? x : -INFINITY;
        sum += exp2(fma(static_cast<double>(x), kLog2eF64, -static_cast<double>(ref)));
        const bool in = x >= thr && x > -INFINITY;
        const unsigned put = __ballot_sync(0xffffffffu, in);
        int at = 0;
        if (lane == 0)
            at = atomicAdd(&count, __popc(put));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(put & ((1u << lane) - 1u));
        if (in && at < kBeamBuf)
            buf[at] = beam_key(x, v);
    }
    if (__any_sync(0xffffffffu, any_bad) && lane == 0 && status)
        atomicOr(status, kBeamDevBadLogit);
    sum = warp_sum(sum);
    if (lane == 0)
        red_sum[warp] = sum;
    __syncthreads();
    const int n = count;
    BeamCand *out = cand + (row * parts + pt) * C;
    int kept;
    if (n <= kBeamBuf) {
        kept = n < C ? n : C;
        for (int i = tid; i < n; i += kBeamThreads) {
            const uint64_t k = buf[i];
            int rank = 0;
            for (int j = 0; j < n; ++j)
                rank += buf[j] > k;
            if (rank < C)
                out[rank] = BeamCand{from_ordered(static_cast<uint32_t>(k >> 32)),
                                     static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(k))};
        }
    } else {
        // more values at the threshold than fit (many equal logits, whose terms
        // all err the same way): the whole sum in FP64, and the best one below the
        // last, C times over the part
        sum = 0.0;
        for (int64_t v0 = begin; v0 < end; v0 += kBeamBatch) {
#pragma unroll 1
            for (int i = 0; i < kBeamPerThread; ++i) {
                const int64_t v = beam_token<T>(v0, i, tid);
                const float x = v < V ? BeamVec<T>::one(x0 + v) : -INFINITY;
                if (x < kBeamMaxLogit)
                    sum += exp2(fma(static_cast<double>(x), kLog2eF64, -static_cast<double>(ref)));
            }
        }
        sum = warp_sum(sum);
        if (lane == 0)
            red_sum[warp] = sum;  // read after the barriers below
        uint64_t last = ~0ull;
        for (kept = 0; kept < C; ++kept) {
            uint64_t b = 0;
            for (int64_t v0 = begin; v0 < end; v0 += kBeamBatch) {
                float x[kBeamPerThread];
                beam_load(x0, v0, V, off, x);
                beam_clean(x);
#pragma unroll
                for (int i = 0; i < kBeamPerThread; ++i) {
                    const uint64_t k = beam_key(x[i], beam_token<T>(v0, i, tid));
                    if (x[i] > -INFINITY && k < last && k > b)
                        b = k;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t c = __shfl_xor_sync(0xffffffffu, b, o);
                b = c > b ? c : b;
            }
            if (lane == 0)
                win[warp] = b;
            __syncthreads();
            b = win[0];
#pragma unroll
            for (int i = 1; i < kBeamWarps; ++i)
                b = win[i] > b ? win[i] : b;
            __syncthreads();
            if (b == 0)
                break;
            last = b;
            if (tid == 0)
                out[kept] = BeamCand{from_ordered(static_cast<uint32_t>(b >> 32)),
                                     static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(b))};
        }
    }
    if (tid == 0) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < kBeamWarps; ++i)
            s += red_sum[i];
        part[row * parts + pt] = BeamPartial{s, ref, kept};
    }
    if (fabsf(ref) > kBeamMaxRef && ref > -INFINITY)
        beam_sum_far(logits, cand, part, V, C, parts, batches, red_sum);
}

struct BeamOut {
    float *cand_score;
    int32_t *cand_beam;
    int64_t *cand_token;
    float *next_score;
    int32_t *next_beam;
    int64_t *next_token;
};

// A candidate of the merge: its total as an unsigned integer of the same order, and
// what decides between equal totals, lower first: beam (6 bits), logit (32, the
// higher first), part (19) and place in its list (7), which order as the token does.
struct BeamKey {
    uint64_t total, at;
};
static_assert(kBeamMaxWidth <= 1 << 6 && kBeamMaxCand <= 1 << 7, "bits of BeamKey::at");

__device__ __forceinline__ uint64_t ordered64(double x)
{
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));  // -0 as 0
    return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}

__device__ __forceinline__ double from_ordered64(uint64_t k)
{
    return __longlong_as_double(static_cast<long long>(k ^ ((k >> 63) ? 0x8000000000000000ull : ~0ull)));
}

__device__ __forceinline__ bool ahead(const BeamKey &a, const BeamKey &b)
{
    return a.total > b.total || (a.total == b.total && a.at < b.at);
}

// One CTA per batch entry.  The candidates of all parts of all beams (a few KB in
// L2) give a threshold, and those that reach it are ranked.
// o.next_score may be `scores`: an entry's are read before any is written.
__global__ void __launch_bounds__(kBeamThreads)
    beam_merge_kernel(const float *scores, const int32_t *__restrict__ done, const BeamPartial *part,
                      const BeamCand *cand, BeamOut o, int32_t W, int32_t C, int32_t parts, int64_t eos,
                      int32_t *status)
{
    // total = (x - base) + off.  off: score - lse, -inf for a beam with no continuation.
    // base: 0, or the row's largest logit beyond kBeamMaxRef, which off then leaves out
    // (lse would swallow the logarithm of the sum).
    __shared__ double off[kBeamMaxWidth];
    __shared__ float base[kBeamMaxWidth];
    __shared__ uint32_t red[kBeamWarps];
    __shared__ BeamKey buf[kBeamBuf];
    __shared__ BeamKey win[kBeamWarps];
    __shared__ BeamKey sorted[kBeamMaxCand];
    __shared__ int32_t buf_tok[kBeamBuf], sorted_tok[kBeamMaxCand];
    __shared__ int count;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t n = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (done && done[n]) {
        // nothing is chosen: every beam stays where it is
        for (int i = tid; i < C; i += kBeamThreads) {
            o.cand_score[n * C + i] = -INFINITY;
            o.cand_beam[n * C + i] = -1;
            o.cand_token[n * C + i] = -1;
        }
        if (o.next_score)
            for (int w = tid; w < W; w += kBeamThreads) {
                o.next_score[n * W + w] = scores[n * W + w];
                o.next_beam[n * W + w] = w;
                o.next_token[n * W + w] = eos < 0 ? 0 : eos;
            }
        return;
    }
    if (tid == 0)
        count = 0;

    const int items = W * parts * C;
    // item i: rank i % C of part (i / C) % parts of beam i / per_row.  What lies past
    // a list's end, or belongs to a beam whose row was not read, is not used.
    struct Raw {
        BeamCand c;
        int32_t w, place;  // place: part << 7 | rank
        bool listed;
    };
    auto fetch = [&](int i) -> Raw {
        const unsigned list = static_cast<unsigned>(i) / static_cast<unsigned>(C);  // of the entry
        const int j = i - static_cast<int>(list) * C;
        const int64_t rc = n * W * parts + list;
        const int32_t w = static_cast<int32_t>(list / static_cast<unsigned>(parts));
        return Raw{cand[rc * C + j], w, (static_cast<int32_t>(list) - w * parts) << 7 | j, j < part[rc].count};
    };
    auto key_of = [&](const Raw &r, BeamKey &k) -> bool {
        if (!(off[r.w] > -INFINITY) || !r.listed)
            return false;
        k.total = ordered64((static_cast<double>(r.c.x) - static_cast<double>(base[r.w])) + off[r.w]);
        k.at = static_cast<uint64_t>(r.w) << 58 | static_cast<uint64_t>(~ordered(r.c.x)) << 26 |
               static_cast<uint32_t>(r.place);
        return k.total >= ordered64(-static_cast<double>(FLT_MAX));  // FP32 has no room for less
    };
    constexpr int HELD = 4;  // candidates a thread keeps, under way while lse is made
    Raw raw[HELD];
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
        const int i = tid + j * kBeamThreads;
        raw[j].listed = false;
        raw[j].w = raw[j].place = 0;
        if (i < items)
            raw[j] = fetch(i);
    }
    // A warp per beam.  Its score and a part per lane are fetched together; parts of
    // beams that were not read hold anything, and are not used.
    for (int w = warp; w < W; w += kBeamWarps) {
        const BeamPartial *pp = part + (n * W + w) * parts;
        const float sc = scores[n * W + w];
        float ref = lane < parts ? pp[lane].ref : -INFINITY;
        double sum = lane < parts ? pp[lane].sum : 0.0;
        double r = -INFINITY;
        float from = 0.f;
        if (beam_live(sc)) {
            float c = ref;
            for (int k = lane + 32; k < parts; k += 32)
                c = fmaxf(c, pp[k].ref);
            c = from_ordered(__reduce_max_sync(0xffffffffu, ordered(c)));
            if (fabsf(c) == FLT_MAX) {
                // sums against the largest logit of each part, the first of its list
                const BeamCand *first = cand + (n * W + w) * parts * C;
                from = -INFINITY;
                for (int k = lane; k < parts; k += 32)
                    if (pp[k].ref == c)
                        from = fmaxf(from, first[static_cast<int64_t>(k) * C].x);
                from = from_ordered(__reduce_max_sync(0xffffffffu, ordered(from)));
                double s = 0.0;
                for (int k = lane; k < parts; k += 32)
                    if (pp[k].ref == c)
                        s += pp[k].sum * exp(static_cast<double>(first[static_cast<int64_t>(k) * C].x) -
                                             static_cast<double>(from));
                r = static_cast<double>(sc) - log(warp_sum(s));
            } else if (c > -INFINITY) {
                double s = ref > -INFINITY ? sum * pow2(ref - c) : 0.0;
                for (int k = lane + 32; k < parts; k += 32) {
                    ref = pp[k].ref;
                    if (ref > -INFINITY)
                        s += pp[k].sum * pow2(ref - c);
                }
                s = warp_sum(s);
                constexpr double kLn2 = 0.69314718055994530942;
                r = static_cast<double>(sc) - (static_cast<double>(c) + log2(s)) * kLn2;
            }
        } else if (lane == 0 && status && !(sc < INFINITY)) {
            atomicOr(status, kBeamDevBadLogit);  // a score of NaN or +inf
        }
        if (lane == 0) {
            off[w] = r;
            base[w] = from;
        }
    }
    __syncthreads();

    // rounded down, so that a thread's maximum is a bound its candidate reaches
    float best = -INFINITY;
    BeamKey k;
#pragma unroll
    for (int j = 0; j < HELD; ++j)
        if (key_of(raw[j], k))
            best = fmaxf(best, __double2float_rd(from_ordered64(k.total)));
    for (int i = tid + HELD * kBeamThreads; i < items; i += kBeamThreads)
        if (key_of(fetch(i), k))
            best = fmaxf(best, __double2float_rd(from_ordered64(k.total)));
    const float thr = block_threshold(best, C, red);
    if (best >= thr && best > -INFINITY) {
        const uint64_t least = ordered64(static_cast<double>(thr));
        auto put = [&](const Raw &r) {
            if (key_of(r, k) && k.total >= least) {
                const int at = atomicAdd(&count, 1);
                if (at < kBeamBuf) {
                    buf[at] = k;
                    buf_tok[at] = r.c.tok;
                }
            }
        };
#pragma unroll
        for (int j = 0; j < HELD; ++j)
            put(raw[j]);
        for (int i = tid + HELD * kBeamThreads; i < items; i += kBeamThreads)
            put(fetch(i));
    }
    __syncthreads();
    const int m = count;
    int kept;
    if (m <= kBeamBuf) {
        kept = m < C ? m : C;
        for (int i0 = 0; i0 < m; i0 += kBeamThreads / 8) {
            const int i = i0 + (tid >> 3);
            const BeamKey c = i < m ? buf[i] : BeamKey{0, 0};
            const int rank = beam_rank(tid & 7, m, [&](int j) { return ahead(buf[j], c); });
            if (i < m && rank < C && (tid & 7) == 0) {
                sorted[rank] = c;
                sorted_tok[rank] = buf_tok[i];
            }
        }
        __syncthreads();
    } else {
        BeamKey last{~0ull, 0};
        for (kept = 0; kept < C; ++kept) {
            BeamKey b{0, ~0ull};
            for (int i = tid; i < items; i += kBeamThreads)
                if (key_of(fetch(i), k) && ahead(last, k) && ahead(k, b))
                    b = k;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) {
                const BeamKey c{__shfl_xor_sync(0xffffffffu, b.total, s),
                                __shfl_xor_sync(0xffffffffu, b.at, s)};
                if (ahead(c, b))
                    b = c;
            }
            if (lane == 0)
                win[warp] = b;
            __syncthreads();
            b = win[0];
            for (int i = 1; i < kBeamWarps; ++i)
                if (ahead(win[i], b))
                    b = win[i];
            __syncthreads();
            if (b.total == 0)
                break;
            last = b;
            if (tid == 0) {
                sorted[kept] = b;
                const int64_t list = (n * W + (b.at >> 58)) * parts + (b.at >> 7 & 0x7ffff);
                sorted_tok[kept] = cand[list * C + (b.at & 127)].tok;
            }
        }
        __syncthreads();
    }
    // One warp writes, 32 candidates at a time: those that go on are numbered by
    // the ones before them.
    if (warp != 0)
        return;
    int gone_on = 0;
    for (int i0 = 0; i0 < C; i0 += 32) {
        const int i = i0 + lane;
        const bool have = i < kept;
        const BeamKey c = have ? sorted[i] : BeamKey{0, 0};
        const int32_t beam = have ? static_cast<int32_t>(c.at >> 58) : -1;
        const int64_t tok = have ? sorted_tok[i] : -1;
        const float sc = have ? static_cast<float>(from_ordered64(c.total)) : -INFINITY;
        if (i < C) {
            o.cand_score[n * C + i] = sc;
            o.cand_beam[n * C + i] = beam;
            o.cand_token[n * C + i] = tok;
        }
        const bool on = have && tok != eos;
        const unsigned all = __ballot_sync(0xffffffffu, on);
        const int place = gone_on + __popc(all & ((1u << lane) - 1u));
        if (o.next_score && on && place < W) {
            o.next_score[n * W + place] = sc;
            o.next_beam[n * W + place] = beam;
            o.next_token[n * W + place] = tok;
        }
        gone_on += __popc(all);
    }
    if (o.next_score)
        // places that no candidate fills: a dead beam that stays where it is
        for (int w = gone_on + lane; w < W; w += 32) {
            o.next_score[n * W + w] = -INFINITY;
            o.next_beam[n * W + w] = w;
            o.next_token[n * W + w] = eos < 0 ? 0 : eos;
        }
}

// ---------------------------------------------------------------- reorder

constexpr int kReorderMaxStates = 128;
constexpr int kReorderThreads = 256;
constexpr int kReorderColumns = 2;  // columns a thread has under way at once

struct ReorderParams {
    uint8_t *state[kReorderMaxStates];
    int64_t entry_stride, beam_stride;  // bytes
    int64_t outer_stride[3];
    uint32_t outer[3];                  // extents (1 where unused)
    uint32_t run_vecs;                  // vectors in the contiguous run
    uint32_t columns;                   // outer[0] * outer[1] * outer[2] * run_vecs
    int32_t W;
    const int32_t *parents;
    int32_t *status;
};

// state[.., n, w, ..] = old state[.., n, parents[n][w], ..], in place: a thread
// owns vector-wide columns of an entry, reads what every beam whose parent
// is another takes over, and only then writes.  No row that stays is touched,
// and a row that several beams take is read from memory once (L1 serves the
// rest), so the traffic is the rows wanted plus the rows changed: bound by HBM (16
// caches of 16 x 4 beams, 2.5 GB moved: 388 us, 6.5 TB/s; a quarter more with one column under way
// per thread instead of two).
// MAXW bounds W at compile time, so that the column's values stay in registers:
// vectors of 16 bytes up to 16 beams, 8 up to 32, 4 up to 64.
template <typename VecT, int MAXW>
__global__ void __launch_bounds__(kReorderThreads)
    beam_reorder_kernel(const __grid_constant__ ReorderParams p)
{
    __shared__ int32_t from[kBeamMaxWidth];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t n = blockIdx.y;
    bool moves = false;
    if (threadIdx.x < p.W) {
        const int w = threadIdx.x;
        int q = p.parents[n * p.W + w];
        if (q < 0 || q >= p.W) {
            if (p.status && blockIdx.x == 0 && blockIdx.z == 0)
                atomicOr(p.status, kBeamDevBadParent);
            q = w;  // the row is left as it is
        }
        from[w] = q;
        moves = q != w;
    }
    if (!__syncthreads_or(moves))
        return;
    uint8_t *base = p.state[blockIdx.z] + n * p.entry_stride;
    constexpr int U = kReorderColumns;
    const uint32_t step = gridDim.x * kReorderThreads;
    for (uint32_t c0 = blockIdx.x * kReorderThreads + threadIdx.x; c0 < p.columns; c0 += U * step) {
        uint8_t *col[U];
        VecT x[U][MAXW];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const uint32_t c = c0 + k * step;
            const uint32_t r = c / p.run_vecs, v = c - r * p.run_vecs;
            const uint32_t r1 = r / p.outer[0], i0 = r - r1 * p.outer[0];
            const uint32_t i2 = r1 / p.outer[1], i1 = r1 - i2 * p.outer[1];
            col[k] = c < p.columns ? base + i0 * p.outer_stride[0] + i1 * p.outer_stride[1] +
                                         i2 * p.outer_stride[2] + static_cast<int64_t>(v) * sizeof(VecT)
                                   : nullptr;
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int w = 0; w < MAXW; ++w)
                if (col[k] && w < p.W && from[w] != w)
                    x[k][w] = *reinterpret_cast<const VecT *>(col[k] + from[w] * p.beam_stride);
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int w = 0; w < MAXW; ++w)
                if (col[k] && w < p.W && from[w] != w)
                    *reinterpret_cast<VecT *>(col[k] + w * p.beam_stride) = x[k][w];
    }
}

}  // namespace lmh
