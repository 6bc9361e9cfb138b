// lora_kernels.cuh -- the skinny products of the low-rank adapters:
//
//   rows   t[i, r]      = sum_c Y[i, c] P_a(r, c)      one row per token: u = s X A^T, g = s dl B
//   cols   D_a[c, r]    = sum_{i of a} Y[i, c] t[i, r] one matrix per adapter: dB = dl^T u, dA = g^T X
//
// Both stream Y (dlogits: 1 GB at 4096 x 128256) through shared memory once with
// cp.async.  With 2 to 12 MMAs per 512 bytes read, mma.sync on register fragments
// nearly keeps up with that stream and needs no tensor memory (rank 32 at that
// size: rows 236-240 us, columns 294-316 us, 4.4 and 3.5 TB/s; the columns' three parts
// keep the mma.sync pipe half busy).
//
//   lora_rows_kernel    64 tokens x a range of c; a partial t per range.  For
//                       each adapter among the tokens the product of all 64 is
//                       formed and the rows of that adapter's tokens are kept.
//   lora_expand_kernel  sums the partials in a fixed order, scales, and writes
//                       t (FP32), its split into BF16 parts for the
//                       GEMM, and the slots of every token tile
//   lora_group_kernel   the tokens of each adapter, in order
//   lora_split_kernel   t in that order as three BF16 parts (FP32's 24 bits)
//   lora_cols_kernel    128 columns of one adapter over its tokens
//
// Sums: FP32 in the MMAs over at most 256 terms, then added rounded to nearest
// (rows: FP64 across ranges).  No atomics on values; every result has one order.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "lora_gemm.cuh"
#include "ptx.cuh"

namespace lmh {

constexpr int kRowsTokens = 64;    // tokens of one lora_rows_kernel CTA
constexpr int kRowsSub = 128;      // columns of Y staged at once
constexpr int kRowsThreads = 128;
constexpr int kRankBlock = 64;     // ranks of one CTA (grid.z takes the others)
constexpr int kColsTile = 128;     // columns of Y of one lora_cols_kernel CTA
constexpr int kColsTokens = 32;    // tokens staged at once
constexpr int kColsThreads = 128;
constexpr int kColsStages = 3;
constexpr int kColsPromote = 8;    // stages (256 tokens) summed in the MMAs
constexpr int kExpandTokens = 4;  // tokens of one lora_expand_kernel CTA, at most
constexpr int kDevBadAdapter = 0x8;  // LMH_DEV_BAD_ADAPTER

// 16 bytes global -> shared; zeros where `in` is false (nothing is read then).
__device__ __forceinline__ void cp16(void *dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void *p)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void *p)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Rows of shared tiles are padded to an odd number of 16-byte units, so that the
// eight rows of an ldmatrix lie in different banks.
constexpr int pad_row(int elems) { return elems * 2 + 16; }

template <bool P_MN, int NT>
struct RowsCfg {
    static constexpr int STAGES = 2;  // blocks under way; a third costs a resident CTA
    static constexpr int RB = NT * 16;
    static constexpr int Y_ROW = pad_row(kRowsSub);
    static constexpr int Y_BYTES = kRowsTokens * Y_ROW;
    static constexpr int P_ROW = P_MN ? pad_row(RB) : pad_row(kRowsSub);
    static constexpr int P_BYTES = (P_MN ? kRowsSub : RB) * P_ROW;
    static constexpr int SMEM = STAGES * (Y_BYTES + P_BYTES);
};

// partial[range][i][r]: the range's share of t.  Y [M][Cdim] BF16; P_MN: P
// [adapter][Cdim][R] (B), else [adapter][R][Cdim] (A).  Rpad: R rounded up to 16.
// grid (ranges of columns, tiles of tokens, rank blocks x slot groups).
//   order (or NULL) gives the tokens adapter by adapter, total[0] of them: a tile
//     then holds one or two adapters instead of as many as 64 tokens in any order
//     have, each of which costs a read of its columns and a product.
//   groups: a tile's adapters are dealt out to so many CTAs, each of which keeps
//     the rows of its own (64 tokens with 28 adapters, K = 4096: 20.2 us without,
//     8.8 us with).
template <bool P_MN, int NT>
__global__ void __launch_bounds__(kRowsThreads)
    lora_rows_kernel(const __nv_bfloat16 *__restrict__ Y, const __nv_bfloat16 *__restrict__ P,
                     const int32_t *__restrict__ adapter, float *__restrict__ partial, int64_t M,
                     int64_t Cdim, int32_t R, int32_t Rpad, int32_t N, int32_t subs_per_range,
                     int32_t groups, const int32_t *__restrict__ order, const int32_t *__restrict__ total)
{
    using G = RowsCfg<P_MN, NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int32_t ids[kRowsTokens];
    __shared__ int32_t toks[kRowsTokens];
    __shared__ int32_t list[kRowsTokens];
    __shared__ int warp_n[2];
    uint8_t *ybuf = smem, *pbuf = smem + G::STAGES * G::Y_BYTES;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kRowsTokens;
    const int r0 = static_cast<int>(blockIdx.z) / groups * kRankBlock;
    const int group = static_cast<int>(blockIdx.z) % groups;
    pdl_wait();
    pdl_launch_dependents();
    bool first = false;
    if (tid < kRowsTokens) {
        const int64_t i = i0 + tid;
        int32_t tok = -1;
        if (order)
            tok = i < *total ? order[i] : -1;
        else if (i < M)
            tok = static_cast<int32_t>(i);
        const int32_t a = tok >= 0 ? adapter[tok] : -1;
        ids[tid] = a < 0 || a >= N ? -1 : a;
        toks[tid] = tok;
    }
    __syncthreads();
    if (tid < kRowsTokens) {
        const int32_t a = ids[tid];
        bool seen = false;
#pragma unroll 16
        for (int j = 0; j < kRowsTokens; ++j)
            seen |= j < tid && ids[j] == a;
        first = a >= 0 && !seen;
        const unsigned b = __ballot_sync(0xffffffffu, first);
        if (lane == 0)
            warp_n[warp] = __popc(b);
    }
    __syncthreads();
    // this CTA's share of the tile's adapters: every groups-th from `group`
    const int nslot = (warp_n[0] + warp_n[1] - group + groups - 1) / groups;
    if (nslot <= 0)
        return;
    if (tid < kRowsTokens) {
        const unsigned b = __ballot_sync(0xffffffffu, first);
        const int slot = (warp ? warp_n[0] : 0) + __popc(b & ((1u << lane) - 1u));
        if (first && slot % groups == group)
            list[slot / groups] = ids[tid];
    }
    __syncthreads();

    const int64_t nsub_all = (Cdim + kRowsSub - 1) / kRowsSub;
    const int64_t sub0 = static_cast<int64_t>(blockIdx.x) * subs_per_range;
    const int nsub = static_cast<int>(nsub_all - sub0 < subs_per_range ? nsub_all - sub0 : subs_per_range);
    float acc[2 * NT][4];
#pragma unroll
    for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[n][e] = 0.f;
    const int steps = nsub * nslot;
    // What a thread copies is the same in every step, up to the columns and the
    // adapter: rows yr, yr + 8, .. of Y at 16-byte unit yc, and P's units tid,
    // tid + 128, ..; addresses are made once.
    const int yr = tid >> 4, yc = tid & 15;
    const __nv_bfloat16 *ysrc[kRowsTokens / 8];
#pragma unroll
    for (int i = 0; i < kRowsTokens / 8; ++i) {
        const int tok = toks[yr + 8 * i];
        ysrc[i] = tok < 0 ? nullptr : Y + static_cast<int64_t>(tok) * Cdim + sub0 * kRowsSub + yc * 8;
    }
    constexpr int UNITS = P_MN ? G::RB / 8 : kRowsSub / 8;  // 16-byte units in a row of P's tile
    int64_t psrc[2 * NT];                                   // from the adapter's first element of this range
    bool prank[2 * NT];                                     // a rank below R
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
        const int k = tid + i * kRowsThreads, row = k / UNITS, ch = k % UNITS;
        if (P_MN) {
            psrc[i] = (sub0 * kRowsSub + row) * R + r0 + ch * 8;
            prank[i] = r0 + ch * 8 < R;
        } else {
            psrc[i] = static_cast<int64_t>(r0 + row) * Cdim + sub0 * kRowsSub + ch * 8;
            prank[i] = r0 + row < R;
        }
    }
    const int64_t pstep = P_MN ? static_cast<int64_t>(kRowsSub) * R : kRowsSub;
    // step: columns `sub` against the tile's adapter j
    int ls = 0, lj = 0, lt = 0;
    auto load = [&]() {
        if (lt < steps) {
            const int64_t left = Cdim - (sub0 + ls) * kRowsSub;  // columns from here to the end
            if (lj == 0) {
                uint8_t *y = ybuf + (ls % G::STAGES) * G::Y_BYTES + yr * G::Y_ROW + yc * 16;
                const bool inc = yc * 8 < left;
#pragma unroll
                for (int i = 0; i < kRowsTokens / 8; ++i) {
                    const bool in = inc && ysrc[i];
                    cp16(y + i * 8 * G::Y_ROW, in ? ysrc[i] + ls * kRowsSub : Y, in);
                }
            }
            uint8_t *pb = pbuf + (lt % G::STAGES) * G::P_BYTES;
            const __nv_bfloat16 *base = P + static_cast<int64_t>(list[lj]) * R * Cdim + ls * pstep;
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                const int k = tid + i * kRowsThreads, row = k / UNITS, ch = k % UNITS;
                const bool in = prank[i] && (P_MN ? row : ch * 8) < left;
                cp16(pb + row * G::P_ROW + ch * 16, in ? base + psrc[i] : P, in);
            }
            if (++lj == nslot) {
                lj = 0;
                ++ls;
            }
            ++lt;
        }
        cp_commit();
    };
    const int g = lane >> 2;  // this thread's rows of the warp's 16: g and g + 8
    const int id0 = ids[warp * 16 + g], id1 = ids[warp * 16 + g + 8];
#pragma unroll
    for (int i = 0; i < G::STAGES - 1; ++i)
        load();
    int sub = 0, j = -1;
    for (int t = 0; t < steps; ++t) {
        cp_wait<G::STAGES - 2>();
        __syncthreads();  // step t has landed; the buffers of step t - 1 are free
        load();
        if (++j == nslot) {
            j = 0;
            ++sub;
        }
        const int a = list[j];
        const bool k0 = id0 == a, k1 = id1 == a;
        if (!__any_sync(0xffffffffu, k0 || k1))
            continue;
        const uint8_t *y = ybuf + (sub % G::STAGES) * G::Y_BYTES;
        const uint8_t *pb = pbuf + (t % G::STAGES) * G::P_BYTES;
        float part[2 * NT][4];
#pragma unroll
        for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part[n][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < kRowsSub / 16; ++ks) {
            uint32_t fa[4];
            ldsm4(fa, y + (warp * 16 + (lane & 15)) * G::Y_ROW + (ks * 16 + (lane >> 4) * 8) * 2);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t fb[4];
                const int mat = lane >> 3, l = lane & 7;
                if (P_MN)
                    ldsm4t(fb, pb + (ks * 16 + (mat & 1) * 8 + l) * G::P_ROW + (n * 16 + (mat >> 1) * 8) * 2);
                else
                    ldsm4(fb, pb + (n * 16 + (mat >> 1) * 8 + l) * G::P_ROW + (ks * 16 + (mat & 1) * 8) * 2);
                mma16816(part[2 * n], fa, fb[0], fb[1]);
                mma16816(part[2 * n + 1], fa, fb[2], fb[3]);
            }
        }
        // only the rows of this adapter's tokens (a select, not a product with
        // zero: another adapter's infinities stay out)
#pragma unroll
        for (int n = 0; n < 2 * NT; ++n) {
            if (k0) {
                acc[n][0] += part[n][0];
                acc[n][1] += part[n][1];
            }
            if (k1) {
                acc[n][2] += part[n][2];
                acc[n][3] += part[n][3];
            }
        }
    }
    cp_wait<0>();
    // rows of tokens without an adapter, and of other groups', are not this CTA's
    bool own0 = false, own1 = false;
    for (int j = 0; j < nslot; ++j) {
        own0 |= id0 == list[j];
        own1 |= id1 == list[j];
    }
    float *out = partial + static_cast<int64_t>(blockIdx.x) * M * Rpad;
    const int64_t ta = toks[warp * 16 + g], tb = toks[warp * 16 + g + 8];
#pragma unroll
    for (int n = 0; n < 2 * NT; ++n) {
        const int r = r0 + n * 8 + (lane & 3) * 2;
        if (r < Rpad) {
            if (own0)
                *reinterpret_cast<float2 *>(out + ta * Rpad + r) = make_float2(acc[n][0], acc[n][1]);
            if (own1)
                *reinterpret_cast<float2 *>(out + tb * Rpad + r) = make_float2(acc[n][2], acc[n][3]);
        }
    }
}

// x as BF16 high part and remainder, the part towards zero: three of them hold FP32's
// 24 bits, and the largest x have a finite one.  An infinite x has no remainder.
__device__ __forceinline__ __nv_bfloat16 split_hi(float x, float &rest)
{
    const __nv_bfloat16 h = __float2bfloat16_rz(x);
    const float hf = __bfloat162float(h);
    rest = fabsf(hf) < INFINITY ? x - hf : 0.f;
    return h;
}

// grid (token tiles of the GEMM, parts of `tokens` tokens).
//   t    [M][R] FP32, scaled: u or g (0 for a token without adapter)
//   ux   (or NULL) [tile][stages][bn][64] BF16: see lora_stages
//   count, slot_table, slot_mask: see LoraParams (written by part 0)
__global__ void __launch_bounds__(256)
    lora_expand_kernel(const float *__restrict__ partial, int32_t ranges, const int32_t *__restrict__ adapter,
                       const float *__restrict__ scale, float *__restrict__ t_out,
                       __nv_bfloat16 *__restrict__ ux, int2 *__restrict__ tile_count,
                       int2 *__restrict__ slot_table, uint32_t *__restrict__ slot_mask, int32_t bn,
                       int32_t slot_stride, int32_t max_slots, int32_t stages, int64_t M, int32_t R,
                       int32_t Rpad, int32_t N, int32_t tokens, int32_t *status)
{
    __shared__ int32_t ids[256];
    __shared__ int32_t warp_n[8];
    __shared__ double share[256];
    extern __shared__ float val[];  // [tokens][Rpad]
    // The GEMM may begin with the shared product at once: all that it reads of that
    // was complete before the row kernel let this one start.
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t tile = blockIdx.x;
    const int64_t i0 = tile * bn;
    const int tok0 = blockIdx.y * tokens;
    if (tid < bn) {
        int32_t a = i0 + tid < M ? adapter[i0 + tid] : -1;
        if (a < -1 || a >= N) {
            if (status && blockIdx.y == 0)
                atomicOr(status, kDevBadAdapter);
            a = -1;
        }
        ids[tid] = a;
    } else if (tid < 256) {
        ids[tid] = -1;
    }
    __syncthreads();

    // Sums over the ranges: `lanes` threads take every lanes-th range of an item
    // (token, rank), and the first of them adds theirs in order.
    const int items = tokens * Rpad;
    const int lanes = items >= 256 ? 1 : 256 / items;
    const int per_pass = 256 / lanes;
    for (int k0 = 0; k0 < items; k0 += per_pass) {
        const int k = k0 + tid % per_pass, q0 = tid / per_pass;
        const int tk = tok0 + k / Rpad, r = k % Rpad;
        const bool in = k < items && q0 < lanes && tk < bn && i0 + tk < M && r < R;
        const int a = in ? ids[tk] : -1;
        double s = 0.0;
        if (a >= 0) {
            const float *p = partial + (i0 + tk) * Rpad + r;
#pragma unroll 8
            for (int q = q0; q < ranges; q += lanes)
                s += static_cast<double>(p[static_cast<int64_t>(q) * M * Rpad]);
        }
        if (lanes > 1) {
            share[tid] = s;
            __syncthreads();
            if (q0 == 0)
                for (int q = 1; q < lanes; ++q)
                    s += share[q * per_pass + tid];
            __syncthreads();
        }
        if (k < items && q0 == 0) {
            const float v = a >= 0 ? static_cast<float>(s * static_cast<double>(scale[a])) : 0.f;
            val[k] = v;
            if (in)
                t_out[(i0 + tk) * R + r] = v;
        }
    }
    __syncthreads();
    // the split parts of this CTA's tokens, eight columns per store
    const int per_token = stages * 8;
    for (int k = tid; ux && k < tokens * per_token; k += 256) {
        const int j = k / per_token, rest = k % per_token;
        const int st = rest >> 3, c0 = (rest & 7) * 8;
        const int tk = tok0 + j;
        if (tk >= bn)
            break;
        int part = st % kSplitParts, r0 = st / kSplitParts * 64 + c0;
        if (R <= 32) {
            const int width = R <= 16 ? 16 : 32;  // columns of a part
            part = st * 2 + c0 / width;
            r0 = c0 % width;
        }
        __nv_bfloat16 h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = r0 + e < Rpad && part < kSplitParts ? val[j * Rpad + r0 + e] : 0.f;
            float rest, rest2;
            const __nv_bfloat16 hi = split_hi(v, rest), mid = split_hi(rest, rest2);
            h[e] = part == 0 ? hi : part == 1 ? mid : __float2bfloat16_rn(rest2);
        }
        *reinterpret_cast<uint4 *>(ux + ((tile * stages + st) * bn + tk) * 64 + c0) = *reinterpret_cast<uint4 *>(h);
    }
    if (blockIdx.y != 0)
        return;
    // The tile's slots, in the order in which their adapters occur: a hash table
    // of the ids, each with its first and last token and the bits of all its tokens.
    constexpr int kBuckets = 512;
    __shared__ int32_t key[kBuckets], lead[kBuckets], tail[kBuckets];
    __shared__ __align__(16) uint32_t bits[kBuckets][kSlotMaskWords];
    __shared__ int32_t spans[256];  // of each slot: first block of 32 tokens | blocks << 4
    for (int k = tid; k < kBuckets; k += 256) {
        key[k] = -1;
        lead[k] = 256;
        tail[k] = 0;
        *reinterpret_cast<uint4 *>(&bits[k][0]) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(&bits[k][4]) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const int32_t a = ids[tid];
    uint32_t h = 0;
    if (a >= 0) {
        h = (static_cast<uint32_t>(a) * 2654435761u) >> 23;
        while (true) {  // at most 256 of the 512 buckets are taken
            const int32_t old = atomicCAS(&key[h], -1, a);
            if (old == -1 || old == a)
                break;
            h = (h + 1) & (kBuckets - 1);
        }
        atomicMin(&lead[h], tid);
        atomicMax(&tail[h], tid);
        atomicOr(&bits[h][warp], 1u << lane);
    }
    __syncthreads();
    const bool first = a >= 0 && lead[h] == tid;
    const unsigned b = __ballot_sync(0xffffffffu, first);
    const unsigned with = __ballot_sync(0xffffffffu, a >= 0);
    if (lane == 0)
        warp_n[warp] = __popc(b) | __popc(with) << 16;
    __syncthreads();
    int slot = __popc(b & ((1u << lane) - 1u)), all = 0, having = 0;
    for (int w = 0; w < 8; ++w) {
        if (w < warp)
            slot += warp_n[w] & 0xffff;
        all += warp_n[w] & 0xffff;
        having += warp_n[w] >> 16;
    }
    if (first) {
        spans[slot] = lead[h] / 32 | (tail[h] / 32 - lead[h] / 32 + 1) << 4;
        slot_table[tile * slot_stride + slot].x = a;
        uint4 *m = reinterpret_cast<uint4 *>(slot_mask + (tile * max_slots + slot) * kSlotMaskWords);
        m[0] = *reinterpret_cast<uint4 *>(&bits[h][0]);
        m[1] = *reinterpret_cast<uint4 *>(&bits[h][4]);
    }
    __syncthreads();
    if (tid != 0)
        return;
    // Pack the spans into accumulators of 256 columns, in order.  The only slot of
    // a tile whose tokens all have it needs none: its span is the whole tile.
    const int64_t rows = M - i0 < bn ? M - i0 : bn;
    int packs = 0;
    if (all == 1 && having == rows) {
        slot_table[tile * slot_stride].y = slot_info(0, 256, 0, 1);
    } else {
        int off = 0;
        for (int s = 0; s < all; ++s) {
            const int lo = (spans[s] & 15) * 32, span = (spans[s] >> 4) * 32;
            const int next = s + 1 < all ? (spans[s + 1] >> 4) * 32 : 512;
            const bool last = off + span + next > 256;
            slot_table[tile * slot_stride + s].y = slot_info(lo, span, off, last);
            off = last ? 0 : off + span;
            packs += last;
        }
    }
    tile_count[tile] = make_int2(all, packs);
}

// One CTA per adapter: start[a] (tokens of lower adapters) and its tokens in
// order, order[start[a] ..].  start has N + 1 entries.
__global__ void __launch_bounds__(1024)
    lora_group_kernel(const int32_t *__restrict__ adapter, int32_t *__restrict__ start,
                      int32_t *__restrict__ order, int64_t M, int32_t N, int32_t *status)
{
    __shared__ int warp_n[32];
    __shared__ int below;
    pdl_wait();
    pdl_launch_dependents();
    const int a = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0)
        below = 0;
    __syncthreads();
    int n = 0;
    for (int64_t i = tid; i < M; i += 1024) {
        const int32_t x = adapter[i];
        n += x >= 0 && x < a;
        if (a == 0 && status && (x < -1 || x >= N))
            atomicOr(status, kDevBadAdapter);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0)
        atomicAdd(&below, n);  // whole numbers: any order
    __syncthreads();
    int at = below;
    if (tid == 0)
        start[a] = at;
    for (int64_t i0 = 0; i0 < M; i0 += 1024) {
        const int64_t i = i0 + tid;
        const bool mine = i < M && adapter[i] == a;
        const unsigned b = __ballot_sync(0xffffffffu, mine);
        if (lane == 0)
            warp_n[warp] = __popc(b);
        __syncthreads();
        int place = __popc(b & ((1u << lane) - 1u)), all = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp)
                place += warp_n[w];
            all += warp_n[w];
        }
        if (mine)
            order[at + place] = static_cast<int32_t>(i);
        at += all;
        __syncthreads();
    }
    if (a == N - 1 && tid == 0)
        start[N] = at;
}

// parts[pos][3][Rpad] BF16 of t[order[pos]]: x = high + middle + low, exact to
// FP32's 24 bits (while the low part stays normal); zeros in the padding.
// grid.y: u, g.
__global__ void __launch_bounds__(256)
    lora_split_kernel(const float *__restrict__ u, const float *__restrict__ g, const int32_t *__restrict__ start,
                      const int32_t *__restrict__ order, __nv_bfloat16 *__restrict__ u_parts,
                      __nv_bfloat16 *__restrict__ g_parts, int32_t N, int32_t R, int32_t Rpad)
{
    pdl_wait();
    pdl_launch_dependents();
    const float *t = blockIdx.y ? g : u;
    __nv_bfloat16 *parts = blockIdx.y ? g_parts : u_parts;
    const int64_t total = static_cast<int64_t>(start[N]) * Rpad;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; k < total;
         k += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t pos = k / Rpad;
        const int r = static_cast<int>(k - pos * Rpad);
        const float x = r < R ? t[static_cast<int64_t>(order[pos]) * R + r] : 0.f;
        float rest, rest2;
        const __nv_bfloat16 h = split_hi(x, rest), m = split_hi(rest, rest2);
        __nv_bfloat16 *o = parts + pos * 3 * Rpad + r;
        o[0] = h;
        o[Rpad] = m;
        o[2 * Rpad] = __float2bfloat16_rn(rest2);
    }
}

template <int NT>
struct ColsCfg {
    static constexpr int RB = NT * 16;
    static constexpr int Y_ROW = pad_row(kColsTile);
    static constexpr int Y_BYTES = kColsTokens * Y_ROW;
    static constexpr int T_ROW = pad_row(3 * RB);
    static constexpr int T_BYTES = kColsTokens * T_ROW;
    static constexpr int SMEM = kColsStages * (Y_BYTES + T_BYTES);
};

// One of the two products of lora_cols_kernel: Y [tokens][Cdim], the parts of t,
// and the output [adapter][Cdim][R], or [adapter][R][Cdim] if `rc`.
struct ColsOp {
    const __nv_bfloat16 *Y;
    const __nv_bfloat16 *parts;
    float *out;
    int64_t Cdim;
    int32_t tiles;
    int32_t rc;
};

// grid (column tiles of dB and then of dA, adapters, rank blocks).  FP32 outputs;
// zeros for an adapter without tokens.
template <int NT>
__global__ void __launch_bounds__(kColsThreads)
    lora_cols_kernel(const ColsOp op_b, const ColsOp op_a, const int32_t *__restrict__ start,
                     const int32_t *__restrict__ order, int32_t R, int32_t Rpad)
{
    const bool is_b = static_cast<int>(blockIdx.x) < op_b.tiles;
    const __nv_bfloat16 *__restrict__ Y = is_b ? op_b.Y : op_a.Y;
    const __nv_bfloat16 *__restrict__ parts = is_b ? op_b.parts : op_a.parts;
    float *__restrict__ out = is_b ? op_b.out : op_a.out;
    const int64_t Cdim = is_b ? op_b.Cdim : op_a.Cdim;
    const bool rc = is_b ? op_b.rc : op_a.rc;
    using G = ColsCfg<NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *ybuf = smem, *tbuf = smem + kColsStages * G::Y_BYTES;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x - (is_b ? 0 : op_b.tiles)) * kColsTile;
    const int a = blockIdx.y, r0 = blockIdx.z * kRankBlock;
    pdl_wait();
    pdl_launch_dependents();
    const int first = start[a], count = start[a + 1] - first;
    const int steps = (count + kColsTokens - 1) / kColsTokens;
    // A thread copies unit yc of rows yr, yr + 8, .. of every stage; their tokens are
    // fetched one stage ahead.
    const int yr = tid >> 4, yc = tid & 15;
    const bool inc = c0 + yc * 8 < Cdim;
    const __nv_bfloat16 *ycol = Y + c0 + yc * 8;
    int tok[kColsTokens / 8];
    auto next_tokens = [&](int t) {
#pragma unroll
        for (int i = 0; i < kColsTokens / 8; ++i) {
            const int pos = t * kColsTokens + yr + 8 * i;
            tok[i] = pos < count ? order[first + pos] : -1;
        }
    };
    next_tokens(0);
    auto load = [&](int t) {
        if (t < steps) {
            uint8_t *y = ybuf + (t % kColsStages) * G::Y_BYTES + yr * G::Y_ROW + yc * 16;
#pragma unroll
            for (int i = 0; i < kColsTokens / 8; ++i) {
                const bool in = inc && tok[i] >= 0;
                cp16(y + i * 8 * G::Y_ROW, in ? ycol + static_cast<int64_t>(tok[i]) * Cdim : Y, in);
            }
            uint8_t *tb = tbuf + (t % kColsStages) * G::T_BYTES;
            const __nv_bfloat16 *src = parts + (static_cast<int64_t>(first) + t * kColsTokens) * 3 * Rpad + r0;
            const int left = count - t * kColsTokens;
            constexpr int UNITS = 3 * (G::RB / 8);
#pragma unroll
            for (int k0 = 0; k0 < kColsTokens * UNITS; k0 += kColsThreads) {
                const int k = k0 + tid;
                const int row = k / UNITS, rest = k % UNITS;
                const int part = rest / (G::RB / 8), ch = rest % (G::RB / 8);
                if (kColsTokens * UNITS % kColsThreads == 0 || k < kColsTokens * UNITS) {
                    const bool in = row < left && r0 + ch * 8 < Rpad;
                    cp16(tb + row * G::T_ROW + (part * G::RB + ch * 8) * 2,
                         in ? src + (row * 3 + part) * Rpad + ch * 8 : parts, in);
                }
            }
            next_tokens(t + 1);
        }
        cp_commit();
    };
    float acc[2][2 * NT][4], part[2][2 * NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[m][n][e] = part[m][n][e] = 0.f;
#pragma unroll
    for (int t = 0; t < kColsStages - 1; ++t)
        load(t);
    const int mat = lane >> 3, l = lane & 7;
    for (int t = 0; t < steps; ++t) {
        cp_wait<kColsStages - 2>();
        __syncthreads();
        load(t + kColsStages - 1);
        const uint8_t *y = ybuf + (t % kColsStages) * G::Y_BYTES;
        const uint8_t *tb = tbuf + (t % kColsStages) * G::T_BYTES;
#pragma unroll
        for (int ks = 0; ks < kColsTokens / 16; ++ks) {
            uint32_t fa[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)  // 16 columns of Y x 16 tokens, out of token-major rows
                ldsm4t(fa[m], y + (ks * 16 + (mat >> 1) * 8 + l) * G::Y_ROW + (warp * 32 + m * 16 + (mat & 1) * 8) * 2);
#pragma unroll
            for (int s = 2; s >= 0; --s) {  // the small parts first
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t fb[4];
                    ldsm4t(fb, tb + (ks * 16 + (mat & 1) * 8 + l) * G::T_ROW + (s * G::RB + n * 16 + (mat >> 1) * 8) * 2);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        mma16816(part[m][2 * n], fa[m], fb[0], fb[1]);
                        mma16816(part[m][2 * n + 1], fa[m], fb[2], fb[3]);
                    }
                }
            }
        }
        if (t % kColsPromote == kColsPromote - 1 || t == steps - 1) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[m][n][e] += part[m][n][e];
                        part[m][n][e] = 0.f;
                    }
        }
    }
    cp_wait<0>();
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
            const int64_t c = c0 + warp * 32 + m * 16 + (lane >> 2) + e2 * 8;
            if (c >= Cdim)
                continue;
#pragma unroll
            for (int n = 0; n < 2 * NT; ++n) {
                const int r = r0 + n * 8 + (lane & 3) * 2;
                if (r >= R)  // R is a multiple of 8: r + 1 < R as well
                    continue;
                const float x = acc[m][n][2 * e2], z = acc[m][n][2 * e2 + 1];
                if (rc) {
                    float *o = out + (static_cast<int64_t>(a) * R + r) * Cdim + c;
                    o[0] = x;
                    o[Cdim] = z;
                } else {
                    *reinterpret_cast<float2 *>(out + (static_cast<int64_t>(a) * Cdim + c) * R + r) = make_float2(x, z);
                }
            }
        }
}

}  // namespace lmh
