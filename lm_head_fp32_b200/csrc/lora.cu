// lora.cu -- C ABI of the LM head with low-rank adapters (declared in
// include/lmhead.h): argument validation, workspace layout, kernel selection
// and launches of lora_kernels.cuh and lora_gemm.cuh.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "lmhead.h"
#include "host.cuh"
#include "lora_gemm.cuh"
#include "lora_kernels.cuh"

namespace {

using namespace lmh::host;
using lmh::GemmCfg;
using lmh::GemmParams;
using lmh::LoraParams;

constexpr int64_t kMaxRank = 256;
constexpr int64_t kMaxAdapters = 65535;              // a grid dimension
constexpr int64_t kMaxTokens = 65535ll * lmh::kRowsTokens;  // likewise
constexpr int64_t kMaxGrouping = int64_t{1} << 34;   // tokens x adapters: the grouping looks at each id per adapter

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Token-tile width of the GEMMs: the smallest supported MMA N that covers M, up
// to 256.
int pick_bn(int64_t M, int least) { return M <= least ? least : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256; }

// Ranges the columns of a row kernel are cut into: enough CTAs that the last ones
// leave few SMs idle (dlogits of 4096 x 128256, rank 32: 424, 296, 253 us with 384,
// 832, 1728), and no more, since each range writes a partial result, which is most of
// the work with few tokens (60 x 792 x 73312, rank 16, both gradients: 74 us with 1480,
// 71 with 740, 72 with 296).
struct RowRanges {
    int64_t subs, ranges, groups;
};
RowRanges row_ranges(int64_t M, int64_t Cdim, int64_t R, int64_t N)
{
    const int64_t nsub = ceil_div(Cdim, lmh::kRowsSub);
    const int64_t base = ceil_div(M, lmh::kRowsTokens) * ceil_div(R, lmh::kRankBlock);
    const int64_t ctas = base < 32 ? 740 : 1480;  // aimed at: five or ten per SM
    int64_t want = ctas / base;
    want = want < 1 ? 1 : want > nsub ? nsub : want;
    const int64_t subs = ceil_div(nsub, want);
    const int64_t ranges = ceil_div(nsub, subs);
    // CTAs still to spare: the adapters of a tile are dealt out to several
    const int64_t most = N < M ? (N < lmh::kRowsTokens ? N : lmh::kRowsTokens) : (M < lmh::kRowsTokens ? M : lmh::kRowsTokens);
    int64_t groups = ctas / (base * ranges);
    groups = groups < 1 ? 1 : groups > most ? most : groups;
    return {subs, ranges, groups};
}

// Whether the row kernel takes the tokens adapter by adapter: where the matrix it
// reads is large, the tokens are more than one tile, and the grouping, which reads
// the ids once per adapter, is small beside it.  (4096 tokens in random order, 8
// adapters of rank 32, dlogits of 128256, the row kernel in its first form: 1.92 ms
// as they come, 0.49 ms grouped, the grouping 7 us; below 64 MB of Y the whole row
// kernel takes no longer than that.)
bool rows_sorted(int64_t M, int64_t Cdim, int64_t N)
{
    return M > lmh::kRowsTokens && N > 1 && M * Cdim >= (int64_t{1} << 25) && N * 64 <= Cdim;
}

int64_t rank_pad(int64_t R) { return (R + 15) / 16 * 16; }

// Byte offsets in the workspace of lmhead_fwd_lora (Cdim = K) and
// lmhead_bwd_dx_lora (Cdim = V).
struct GemmSpace {
    int64_t partial, ux, count, slot, slot_mask, start, order, bytes;
    int64_t tiles, stages, max_slots, slot_stride;
};
GemmSpace gemm_space(int64_t M, int64_t Cdim, int64_t R, int64_t N, int bn)
{
    GemmSpace g;
    g.tiles = ceil_div(M, bn);
    g.stages = lmh::lora_stages(static_cast<int>(R));
    g.max_slots = N < bn ? N : bn;
    g.slot_stride = (g.max_slots + 1) / 2 * 2;
    g.partial = 0;
    g.ux = align256(row_ranges(M, Cdim, R, N).ranges * M * rank_pad(R) * 4);
    g.count = g.ux + align256(g.tiles * g.stages * bn * 128);
    g.slot = g.count + align256(g.tiles * 8);
    g.slot_mask = g.slot + align256(g.tiles * g.slot_stride * 8);
    g.start = g.slot_mask + align256(g.tiles * g.max_slots * lmh::kSlotMaskWords * 4);
    g.order = g.start + align256((N + 1) * 4);
    g.bytes = g.order + align256(M * 4);
    return g;
}

// Byte offsets in the workspace of lmhead_bwd_lora.
struct GradSpace {
    int64_t start, order, u_parts, g_parts, bytes;
};
GradSpace grad_space(int64_t M, int64_t R, int64_t N)
{
    GradSpace g;
    g.start = 0;
    g.order = align256((N + 1) * 4);
    g.u_parts = g.order + align256(M * 4);
    const int64_t parts = align256(M * 3 * rank_pad(R) * 2);
    g.g_parts = g.u_parts + parts;
    g.bytes = g.g_parts + parts;
    return g;
}

// How the tiles are split along the reduction.  Either every tile into `parts` parts
// of `part_kb` k-blocks, or (dX) `tiles` tiles of the last wave in two, each unit (CTA
// pair) that the wave leaves idle taking `rounds` short parts: as lmhead_bwd_dx, where
// that rule is explained and measured.
struct Split {
    int64_t parts = 0, part_kb = 0;
    int64_t tiles = 0, kb = 0, rounds = 0;
    int64_t scratch = 0;  // bytes
};
// Fewer tiles than units: the number of parts that takes the least time, counted in
// k-blocks on the busiest unit, each part with what handing it over costs (about 3 us
// for the 256 KB of a pair's tile, a k-block 0.3 us; narrow tiles less) and `join` for
// the second kernel.  (Logits of 2 x 4096 x 4096 18 us against 27, 300 x 4096 x 4096 40
// against 43, 64 x 4096 x 5000 27 against 35; both gradients of 60 x 792 x 73312 71 us
// against 445, 32 x 2048 x 128256 135 against 735, 256 x 4096 x 128256 310 against 480.)
Split split_all(int64_t tiles, int64_t units, int64_t num_kb, int64_t bn, int64_t tile_m, int64_t join)
{
    Split s;
    const int64_t cost = bn == 256 ? 20 : bn == 128 ? 16 : 8;
    int64_t best = num_kb;
    for (int64_t n = 2; n * 8 <= num_kb && n * tiles <= 2 * units; ++n) {
        const int64_t kb = ceil_div(ceil_div(num_kb, n), 8) * 8, parts = ceil_div(num_kb, kb);
        const int64_t t = ceil_div(tiles * parts, units) * (kb + cost) + join;
        if (parts > 1 && t < best) {
            best = t;
            s.parts = parts;
            s.part_kb = kb;
        }
    }
    if (s.parts > 0)
        s.scratch = tiles * lmh::split_slabs(static_cast<int>(bn), static_cast<int>(s.parts)) * bn * tile_m * 4;
    return s;
}

constexpr int64_t kJoinKb = 8;  // the second kernel, in k-blocks
Split fwd_split(int64_t M, int64_t K, int64_t V)
{
    const int64_t bn = pick_bn(M, 16), tile_m = bn == 256 ? 256 : 128;
    if (V < tile_m)
        return {};
    const int64_t units = num_sms() / (tile_m / 128), tiles = ceil_div(V, tile_m) * ceil_div(M, bn);
    return tiles <= units ? split_all(tiles, units, ceil_div(K, lmh::kBlockK), bn, tile_m, kJoinKb) : Split{};
}

constexpr int64_t kMaxSplitRounds = 8;
Split dx_split(int64_t M, int64_t K, int64_t V)
{
    const int64_t bn = pick_bn(M, 64), tile_m = bn == 256 && K >= 256 ? 256 : 128;
    const int64_t units = num_sms() / (tile_m / 128), tiles = ceil_div(K, tile_m) * ceil_div(M, bn);
    const int64_t num_kb = ceil_div(V, lmh::kBlockK);
    if (tiles <= units)
        return split_all(tiles, units, num_kb, bn, tile_m, kJoinKb);
    Split s;
    if (tile_m != 256)
        return s;
    const int64_t rem = tiles % units;
    if (num_kb < 2 || rem == 0)
        return s;
    const int64_t spare = units - rem, k = ceil_div(rem, spare);
    const int64_t B = (num_kb * k + k) / (k + 1);  // ceil(num_kb k / (k + 1))
    const int64_t span = B > k * (num_kb - B) ? B : k * (num_kb - B);
    if (k <= kMaxSplitRounds && B < num_kb && 10 * span <= 9 * num_kb) {
        s.tiles = rem;
        s.kb = B;
        s.rounds = k;
        s.scratch = rem * 2 * 256 * 256 * 4;
    }
    return s;
}

bool lora_dims_ok(int64_t M, int64_t K, int64_t V, int64_t R, int64_t N)
{
    return dims_ok(M, K, V) && M <= kMaxTokens && R >= 1 && R <= kMaxRank && N >= 1 && N <= kMaxAdapters &&
           M * N <= kMaxGrouping;
}

// 3-D BF16 tensor [outer][mid][inner] (contiguous), 128-byte swizzled boxes of
// 64 x box_mid; out-of-range elements read as zero.
bool make_map3(CUtensorMap *map, const void *base, uint64_t inner, uint64_t mid, uint64_t outer, uint32_t box_mid)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    const cuuint64_t dims[3] = {inner, mid, outer};
    const cuuint64_t strides[2] = {inner * 2, inner * mid * 2};
    const cuuint32_t box[3] = {64, box_mid, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared memory above 48 KB, once per kernel and device.
template <typename K>
lmh_status_t allow_smem(K kern, int bytes, std::atomic<uint64_t> &set)
{
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (set.load() & bit)
        return LMH_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess)
        return LMH_ERR_CUDA;
    set.fetch_or(bit);
    return LMH_OK;
}

struct AdapterOperands {
    const void *base;         // [N][mid][inner] BF16
    uint64_t inner, mid, N;
    const void *ux;           // the split u of every token tile
    uint64_t ux_rows;
    float *scratch;           // the parts of split tiles
};

template <int BN, bool A_MN, typename OutT, bool TMA_STORE, bool PAIR, int RES, bool SPLIT = A_MN>
lmh_status_t launch_impl(const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &tc, const CUtensorMap &ts,
                         const CUtensorMap &tu, const CUtensorMap &tp, GemmParams p, const LoraParams &q,
                         cudaStream_t stream)
{
    constexpr int EW = lmh::lora_epi_warps(BN);
    using C = GemmCfg<BN, A_MN, false, PAIR, RES, EW>;
    auto kern = lmh::lora_gemm_kernel<BN, A_MN, OutT, TMA_STORE, PAIR, RES, EW, SPLIT>;
    static std::atomic<uint64_t> set{0};
    if (const lmh_status_t r = allow_smem(kern, C::SMEM_BYTES, set); r != LMH_OK)
        return r;
    p.wait_limit_ns = lmh::kWaitLimitNs;
    p.num_m_tiles = static_cast<int32_t>(ceil_div(p.Mdim, C::TILE_M));
    p.num_n_tiles = static_cast<int32_t>(ceil_div(p.Ndim, BN));
    const int64_t tiles = static_cast<int64_t>(p.num_m_tiles) * p.num_n_tiles;
    if (tiles > kMaxDim)
        return LMH_ERR_INVALID_ARG;
    const int64_t ctas = num_sms() / C::CTAS;
    const int64_t items = q.split_parts > 0 ? tiles * q.split_parts
                          : p.split_tiles > 0 ? tiles - p.split_tiles + ctas * p.split_rounds : tiles;
    const int64_t units = RES == 1 ? ctas : items;
    const int grid = static_cast<int>((items < units ? items : units) * C::CTAS);
    return launch_ex(kern, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES, stream, PAIR ? 2u : 1u, ta, tb, tc, ts,
                     tu, tp, p, q);
}

// A: the shared weights [outer][inner], MN-major (dX) or K-major; B: [Ndim][Kdim].
// SPLIT: see lora_gemm_kernel.
template <int BN, bool A_MN, typename OutT, bool PAIR, int RES = 1, bool SPLIT = A_MN>
lmh_status_t launch_lora(const void *a, uint64_t a_inner, uint64_t a_outer, const void *b, const AdapterOperands &ad,
                         GemmParams p, const LoraParams &q, cudaStream_t stream)
{
    using C = GemmCfg<BN, A_MN, false, PAIR, RES, lmh::lora_epi_warps(BN)>;
    CUtensorMap ta, tb, tc, ts, tu, tp;
    if (!make_map(&ta, a, a_inner, a_outer, 64, A_MN ? lmh::kBlockK : lmh::kBlockM) ||
        !make_map(&tb, b, static_cast<uint64_t>(p.Kdim), static_cast<uint64_t>(p.Ndim), lmh::kBlockK, C::BN_CTA))
        return LMH_ERR_CUDA;
    std::memset(&ts, 0, sizeof ts);
    std::memset(&tu, 0, sizeof tu);
    if (BN > 128 && (!make_map3(&ts, ad.base, ad.inner, ad.mid, ad.N, A_MN ? lmh::kBlockK : lmh::kBlockM) ||
                     !make_map(&tu, ad.ux, 64, ad.ux_rows, 64, C::BN_CTA)))
        return LMH_ERR_CUDA;
    std::memset(&tp, 0, sizeof tp);
    // split tiles and their parts
    const int64_t split = q.split_parts > 0 ? ceil_div(p.Mdim, C::TILE_M) * ceil_div(p.Ndim, BN) : p.split_tiles;
    const int64_t parts = q.split_parts > 0 ? lmh::split_slabs(BN, q.split_parts) : 2;
    if (split > 0 && !make_out_map(&tp, ad.scratch, false, C::TILE_M, static_cast<uint64_t>(split * parts * BN),
                                   C::TILE_M, C::EPI_CHUNK))
        return LMH_ERR_CUDA;
    const bool tma = make_out_map(&tc, p.out, sizeof(OutT) == 2, static_cast<uint64_t>(p.Mdim),
                                  static_cast<uint64_t>(p.Ndim), static_cast<uint64_t>(p.ldo), C::EPI_CHUNK);
    lmh_status_t r;
    if constexpr (SPLIT && !A_MN) {
        // logits: no tile is stored whole
        r = launch_impl<BN, false, float, true, PAIR, RES, true>(ta, tb, tp, ts, tu, tp, p, q, stream);
    } else if (tma) {
        r = launch_impl<BN, A_MN, OutT, true, PAIR, RES>(ta, tb, tc, ts, tu, tp, p, q, stream);
    } else {
        if constexpr (A_MN)
            return LMH_ERR_MISALIGNED;  // dX rows are multiples of 16 bytes and its base is checked
        std::memset(&tc, 0, sizeof tc);
        r = launch_impl<BN, A_MN, OutT, A_MN, PAIR, RES>(ta, tb, tc, ts, tu, tp, p, q, stream);
    }
    if (r != LMH_OK || split == 0)
        return r;
    p.num_m_tiles = static_cast<int32_t>(ceil_div(p.Mdim, C::TILE_M));
    p.num_n_tiles = static_cast<int32_t>(ceil_div(p.Ndim, BN));
    const int64_t whole = static_cast<int64_t>(p.num_m_tiles) * p.num_n_tiles - split;
    return launch_ex(lmh::lora_join_kernel<OutT>, dim3(static_cast<unsigned>(split), BN / lmh::kJoinRows), dim3(256), 0,
                     stream, 1u, static_cast<const float *>(ad.scratch), static_cast<OutT *>(p.out), p,
                     static_cast<int32_t>(whole), static_cast<int32_t>(parts), BN, C::TILE_M);
}

template <bool P_MN, int NT>
lmh_status_t launch_rows(const void *Y, const void *P, const int32_t *adapter, float *partial, int64_t M, int64_t Cdim,
                         int64_t R, int64_t N, const RowRanges &rr, const int32_t *order, const int32_t *total,
                         cudaStream_t s)
{
    using G = lmh::RowsCfg<P_MN, NT>;
    auto kern = lmh::lora_rows_kernel<P_MN, NT>;
    static std::atomic<uint64_t> set{0};
    if (const lmh_status_t r = allow_smem(kern, G::SMEM, set); r != LMH_OK)
        return r;
    return launch_ex(kern,
                     dim3(static_cast<unsigned>(rr.ranges), static_cast<unsigned>(ceil_div(M, lmh::kRowsTokens)),
                          static_cast<unsigned>(ceil_div(R, lmh::kRankBlock) * rr.groups)),
                     dim3(lmh::kRowsThreads), G::SMEM, s, 1u, static_cast<const __nv_bfloat16 *>(Y),
                     static_cast<const __nv_bfloat16 *>(P), adapter, partial, M, Cdim, static_cast<int32_t>(R),
                     static_cast<int32_t>(rank_pad(R)), static_cast<int32_t>(N), static_cast<int32_t>(rr.subs),
                     static_cast<int32_t>(rr.groups), order, total);
}

// t = s Y P_a over Cdim, its split and the slots of the token tiles, into the
// workspace and t_out.
template <bool P_MN>
lmh_status_t run_rows(const void *Y, const void *P, const float *scale, const int32_t *adapter, float *t_out,
                      uint8_t *ws, const GemmSpace &g, int bn, int64_t M, int64_t Cdim, int64_t R, int64_t N,
                      int32_t *status, cudaStream_t s)
{
    const RowRanges rr = row_ranges(M, Cdim, R, N);
    float *partial = reinterpret_cast<float *>(ws + g.partial);
    int32_t *order = nullptr, *total = nullptr;
    lmh_status_t r = LMH_OK;
    if (rows_sorted(M, Cdim, N)) {
        int32_t *start = reinterpret_cast<int32_t *>(ws + g.start);
        order = reinterpret_cast<int32_t *>(ws + g.order);
        total = start + N;
        r = launch_ex(lmh::lora_group_kernel, dim3(static_cast<unsigned>(N)), dim3(1024), 0, s, 1u, adapter, start,
                      order, M, static_cast<int32_t>(N), static_cast<int32_t *>(nullptr));
        if (r != LMH_OK)
            return r;
    }
    const int64_t nt = R > 48 ? 4 : rank_pad(R) / 16;
    switch (nt) {
    case 1: r = launch_rows<P_MN, 1>(Y, P, adapter, partial, M, Cdim, R, N, rr, order, total, s); break;
    case 2: r = launch_rows<P_MN, 2>(Y, P, adapter, partial, M, Cdim, R, N, rr, order, total, s); break;
    case 3: r = launch_rows<P_MN, 3>(Y, P, adapter, partial, M, Cdim, R, N, rr, order, total, s); break;
    default: r = launch_rows<P_MN, 4>(Y, P, adapter, partial, M, Cdim, R, N, rr, order, total, s); break;
    }
    if (r != LMH_OK)
        return r;
    // few tokens and many ranges: a CTA per token, whose threads share the ranges
    const int64_t tokens = bn <= 128 && rr.ranges > 64 ? 1 : lmh::kExpandTokens;
    return launch_ex(lmh::lora_expand_kernel,
                     dim3(static_cast<unsigned>(g.tiles), static_cast<unsigned>(ceil_div(bn, tokens))),
                     dim3(256), tokens * rank_pad(R) * sizeof(float), s, 1u,
                     static_cast<const float *>(partial), static_cast<int32_t>(rr.ranges), adapter, scale, t_out,
                     bn > 128 ? reinterpret_cast<__nv_bfloat16 *>(ws + g.ux) : nullptr,
                     reinterpret_cast<int2 *>(ws + g.count), reinterpret_cast<int2 *>(ws + g.slot),
                     reinterpret_cast<uint32_t *>(ws + g.slot_mask),
                     static_cast<int32_t>(bn), static_cast<int32_t>(g.slot_stride), static_cast<int32_t>(g.max_slots),
                     static_cast<int32_t>(g.stages), M, static_cast<int32_t>(R), static_cast<int32_t>(rank_pad(R)),
                     static_cast<int32_t>(N), static_cast<int32_t>(tokens), status);
}

LoraParams lora_params(uint8_t *ws, const GemmSpace &g, int64_t R, const void *adapters, const float *t)
{
    LoraParams q{};
    q.adapters = static_cast<const __nv_bfloat16 *>(adapters);
    q.t = t;
    q.count = reinterpret_cast<const int2 *>(ws + g.count);
    q.slot = reinterpret_cast<const int2 *>(ws + g.slot);
    q.slot_mask = reinterpret_cast<const uint32_t *>(ws + g.slot_mask);
    q.slot_stride = static_cast<int32_t>(g.slot_stride);
    q.max_slots = static_cast<int32_t>(g.max_slots);
    q.stages_per_slot = static_cast<int32_t>(g.stages);
    q.rank = static_cast<int32_t>(R);
    return q;
}

template <int NT>
lmh_status_t launch_cols(const lmh::ColsOp &b, const lmh::ColsOp &a, const int32_t *start, const int32_t *order,
                         int64_t R, int64_t N, cudaStream_t s)
{
    using G = lmh::ColsCfg<NT>;
    auto kern = lmh::lora_cols_kernel<NT>;
    static std::atomic<uint64_t> set{0};
    if (const lmh_status_t r = allow_smem(kern, G::SMEM, set); r != LMH_OK)
        return r;
    return launch_ex(kern,
                     dim3(static_cast<unsigned>(b.tiles + a.tiles), static_cast<unsigned>(N),
                          static_cast<unsigned>(ceil_div(R, lmh::kRankBlock))),
                     dim3(lmh::kColsThreads), G::SMEM, s, 1u, b, a, start, order, static_cast<int32_t>(R),
                     static_cast<int32_t>(rank_pad(R)));
}

// SPLIT: the tiles are split along K.
template <typename OutT, bool SPLIT>
lmh_status_t dispatch_fwd(int bn, bool pair, const void *W, uint64_t K, uint64_t V, const void *X,
                          const AdapterOperands &ad, const GemmParams &p, const LoraParams &q, cudaStream_t s)
{
    switch (bn) {
    // one token tile: bound by W.  Two CTAs resident per SM where tensor memory has
    // room for both
    case 16: return launch_lora<16, false, OutT, false, 2, SPLIT>(W, K, V, X, ad, p, q, s);
    case 32: return launch_lora<32, false, OutT, false, 2, SPLIT>(W, K, V, X, ad, p, q, s);
    case 64: return launch_lora<64, false, OutT, false, 2, SPLIT>(W, K, V, X, ad, p, q, s);
    case 128: return launch_lora<128, false, OutT, false, 1, SPLIT>(W, K, V, X, ad, p, q, s);
    default:
        if constexpr (!SPLIT)  // a split one is at least 256 wide
            if (!pair)
                return launch_lora<256, false, OutT, false>(W, K, V, X, ad, p, q, s);
        return launch_lora<256, false, OutT, true, 1, SPLIT>(W, K, V, X, ad, p, q, s);
    }
}

template <typename OutT>
lmh_status_t dispatch_dx(int bn, bool pair, const void *W, uint64_t K, uint64_t V, const void *dl,
                         const AdapterOperands &ad, const GemmParams &p, const LoraParams &q, cudaStream_t s)
{
    switch (bn) {
    case 64: return launch_lora<64, true, OutT, false>(W, K, V, dl, ad, p, q, s);
    case 128: return launch_lora<128, true, OutT, false>(W, K, V, dl, ad, p, q, s);
    default:
        return pair ? launch_lora<256, true, OutT, true>(W, K, V, dl, ad, p, q, s)
                    : launch_lora<256, true, OutT, false>(W, K, V, dl, ad, p, q, s);
    }
}

}  // namespace

extern "C" {

int64_t lmhead_lora_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t R, int64_t N)
{
    if (!lora_dims_ok(M, K, V, R, N))
        return -1;
    const int64_t f = gemm_space(M, K, R, N, pick_bn(M, 16)).bytes + fwd_split(M, K, V).scratch;
    const int64_t d = gemm_space(M, V, R, N, pick_bn(M, 64)).bytes + dx_split(M, K, V).scratch;
    const int64_t w = grad_space(M, R, N).bytes;
    const int64_t fd = f > d ? f : d;
    return fd > w ? fd : w;
}

lmh_status_t lmhead_fwd_lora(const void *X, const void *W, const void *A, const void *B, const float *scale,
                             const int32_t *adapter, float *u, void *logits, int32_t out_dtype, void *workspace,
                             int64_t workspace_bytes, int64_t M, int64_t K, int64_t V, int64_t R, int64_t N,
                             int32_t *status, lmh_stream_t stream)
{
    if (!X || !W || !A || !B || !scale || !adapter || !u || !logits || !workspace || !lora_dims_ok(M, K, V, R, N))
        return LMH_ERR_INVALID_ARG;
    if (bad_dtype(out_dtype))
        return LMH_ERR_UNSUPPORTED;
    if (K % 8 || R % 8 || !aligned(X, 16) || !aligned(W, 16) || !aligned(A, 16) || !aligned(B, 16) ||
        !aligned(scale, 4) || !aligned(adapter, 4) || !aligned(u, 16) || !aligned(workspace, 256) ||
        !aligned(logits, out_dtype == LMH_F32 ? 4 : 2))
        return LMH_ERR_MISALIGNED;
    const int bn = pick_bn(M, 16);
    const GemmSpace g = gemm_space(M, K, R, N, bn);
    const Split split = fwd_split(M, K, V);
    if (workspace_bytes < g.bytes + split.scratch)
        return LMH_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const lmh_status_t r = run_rows<false>(X, A, scale, adapter, u, ws, g, bn, M, K, R, N, status, s);
    if (r != LMH_OK)
        return r;
    GemmParams p{};
    p.out = logits;
    p.ldo = V;
    p.Mdim = static_cast<int32_t>(V);
    p.Ndim = static_cast<int32_t>(M);
    p.Kdim = static_cast<int32_t>(K);
    p.m_fastest = 0;             // consecutive tiles share one W panel
    p.l2_a = M <= bn ? 1 : 0;    // as lmhead_fwd: streamed once with one token tile
    p.l2_b = 2;
    p.l2_out = 1;
    p.status = status;
    const AdapterOperands ad{B, static_cast<uint64_t>(R), static_cast<uint64_t>(V), static_cast<uint64_t>(N),
                             ws + g.ux, static_cast<uint64_t>(g.tiles * g.stages * bn),
                             reinterpret_cast<float *>(ws + g.bytes)};
    LoraParams q = lora_params(ws, g, R, B, u);
    q.split_parts = static_cast<int32_t>(split.parts);
    q.part_kb = static_cast<int32_t>(split.part_kb);
    q.scratch = ad.scratch;
    const bool pair = V >= 256;
    const uint64_t k = static_cast<uint64_t>(K), v = static_cast<uint64_t>(V);
    if (split.parts > 0)
        return out_dtype == LMH_F32 ? dispatch_fwd<float, true>(bn, pair, W, k, v, X, ad, p, q, s)
                                    : dispatch_fwd<__nv_bfloat16, true>(bn, pair, W, k, v, X, ad, p, q, s);
    return out_dtype == LMH_F32 ? dispatch_fwd<float, false>(bn, pair, W, k, v, X, ad, p, q, s)
                                : dispatch_fwd<__nv_bfloat16, false>(bn, pair, W, k, v, X, ad, p, q, s);
}

lmh_status_t lmhead_bwd_dx_lora(const void *dlogits, const void *W, const void *A, const void *B, const float *scale,
                                const int32_t *adapter, float *g_out, void *dX, int32_t out_dtype, void *workspace,
                                int64_t workspace_bytes, int64_t M, int64_t K, int64_t V, int64_t R, int64_t N,
                                int32_t *status, lmh_stream_t stream)
{
    if (!dlogits || !W || !A || !B || !scale || !adapter || !g_out || !dX || !workspace ||
        !lora_dims_ok(M, K, V, R, N))
        return LMH_ERR_INVALID_ARG;
    if (bad_dtype(out_dtype))
        return LMH_ERR_UNSUPPORTED;
    if (K % 8 || V % 8 || R % 8 || !aligned(dlogits, 16) || !aligned(W, 16) || !aligned(A, 16) || !aligned(B, 16) ||
        !aligned(scale, 4) || !aligned(adapter, 4) || !aligned(g_out, 16) || !aligned(dX, 16) ||
        !aligned(workspace, 256))
        return LMH_ERR_MISALIGNED;
    const int bn = pick_bn(M, 64);
    const GemmSpace g = gemm_space(M, V, R, N, bn);
    const Split split = dx_split(M, K, V);
    if (workspace_bytes < g.bytes + split.scratch)
        return LMH_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const lmh_status_t r = run_rows<true>(dlogits, B, scale, adapter, g_out, ws, g, bn, M, V, R, N, status, s);
    if (r != LMH_OK)
        return r;
    GemmParams p{};
    p.out = dX;
    p.ldo = K;
    p.Mdim = static_cast<int32_t>(K);
    p.Ndim = static_cast<int32_t>(M);
    p.Kdim = static_cast<int32_t>(V);
    p.m_fastest = 1;
    p.l2_a = 2;  // as lmhead_bwd_dx
    p.l2_b = 2;
    p.status = status;
    p.split_tiles = static_cast<int32_t>(split.tiles);
    p.split_kb = static_cast<int32_t>(split.kb);
    p.split_rounds = static_cast<int32_t>(split.rounds);
    const AdapterOperands ad{A, static_cast<uint64_t>(K), static_cast<uint64_t>(R), static_cast<uint64_t>(N),
                             ws + g.ux, static_cast<uint64_t>(g.tiles * g.stages * bn),
                             reinterpret_cast<float *>(ws + g.bytes)};
    LoraParams q = lora_params(ws, g, R, A, g_out);
    q.split_parts = static_cast<int32_t>(split.parts);
    q.part_kb = static_cast<int32_t>(split.part_kb);
    q.scratch = ad.scratch;
    const bool pair = K >= 256;
    const uint64_t k = static_cast<uint64_t>(K), v = static_cast<uint64_t>(V);
    return out_dtype == LMH_F32 ? dispatch_dx<float>(bn, pair, W, k, v, dlogits, ad, p, q, s)
                                : dispatch_dx<__nv_bfloat16>(bn, pair, W, k, v, dlogits, ad, p, q, s);
}

lmh_status_t lmhead_bwd_lora(const void *dlogits, const void *X, const float *u, const float *g_in,
                             const int32_t *adapter, float *dA, float *dB, void *workspace, int64_t workspace_bytes,
                             int64_t M, int64_t K, int64_t V, int64_t R, int64_t N, int32_t *status,
                             lmh_stream_t stream)
{
    if (!dlogits || !X || !u || !g_in || !adapter || !dA || !dB || !workspace || !lora_dims_ok(M, K, V, R, N))
        return LMH_ERR_INVALID_ARG;
    if (K % 8 || V % 8 || R % 8 || !aligned(dlogits, 16) || !aligned(X, 16) || !aligned(u, 4) || !aligned(g_in, 4) ||
        !aligned(adapter, 4) || !aligned(dA, 16) || !aligned(dB, 16) || !aligned(workspace, 256))
        return LMH_ERR_MISALIGNED;
    const GradSpace g = grad_space(M, R, N);
    if (workspace_bytes < g.bytes)
        return LMH_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int32_t *start = reinterpret_cast<int32_t *>(ws + g.start), *order = reinterpret_cast<int32_t *>(ws + g.order);
    __nv_bfloat16 *up = reinterpret_cast<__nv_bfloat16 *>(ws + g.u_parts);
    __nv_bfloat16 *gp = reinterpret_cast<__nv_bfloat16 *>(ws + g.g_parts);
    const int32_t r32 = static_cast<int32_t>(R), pad = static_cast<int32_t>(rank_pad(R)), n32 = static_cast<int32_t>(N);
    lmh_status_t r = launch_ex(lmh::lora_group_kernel, dim3(static_cast<unsigned>(N)), dim3(1024), 0, s, 1u, adapter,
                               start, order, M, n32, status);
    const int64_t blocks = ceil_div(M * pad, 256);
    if (r == LMH_OK)
        r = launch_ex(lmh::lora_split_kernel, dim3(static_cast<unsigned>(blocks < 592 ? blocks : 592), 2), dim3(256),
                      0, s, 1u, u, g_in, static_cast<const int32_t *>(start), static_cast<const int32_t *>(order),
                      up, gp, n32, r32, pad);
    if (r != LMH_OK)
        return r;
    const lmh::ColsOp b{static_cast<const __nv_bfloat16 *>(dlogits), up, dB, V,
                        static_cast<int32_t>(ceil_div(V, lmh::kColsTile)), 0};
    const lmh::ColsOp a{static_cast<const __nv_bfloat16 *>(X), gp, dA, K,
                        static_cast<int32_t>(ceil_div(K, lmh::kColsTile)), 1};
    switch (R > 48 ? 4 : rank_pad(R) / 16) {
    case 1: r = launch_cols<1>(b, a, start, order, R, N, s); break;
    case 2: r = launch_cols<2>(b, a, start, order, R, N, s); break;
    case 3: r = launch_cols<3>(b, a, start, order, R, N, s); break;
    default: r = launch_cols<4>(b, a, start, order, R, N, s); break;
    }
    return r;
}

}  // extern "C"
