// lora_gemm.cuh -- the LM head's products with low-rank adapters beside the
// shared weights, as one tcgen05 kernel:
//
//   logits[i, v] = sum_k X[i,k] W[v,k]  + sum_r u[i,r] B_a[v,r]      (A = W,   K-major)
//   dX[i, k]     = sum_v dl[i,v] W[v,k] + sum_r g[i,r] A_a[r,k]      (A = W^T, MN-major)
//
// with a = the token's adapter.  The adapters' term goes into the same sums:
// after the k-blocks of the shared product, each output tile takes one more
// k-block (up to three per 64 ranks) per adapter that occurs among its tokens
// ("slot").  So the delta never travels to memory and back: separate from the
// product it would read and write all logits once more (4.2 GB at 4096 x
// 128256).  u is FP32, the tensor cores take BF16: it is split into three parts (FP32's
// 24 bits; two, 2^-18 of u, leave an error of 1.1e-6 of the logits' norm where the term
// is as large as the rest), B_a entering three times.  For a BF16 output too: rounded
// to BF16, u would lose 2^-9 of the term, many of the output's steps where the term
// and the rest cancel.
//
// A slot's product is formed for the 32-aligned span of its tokens, and the
// epilogue adds the columns of those tokens alone: an adapter that holds
// infinities or NaN reaches no other request's tokens, as a product with zeros
// would.  The slots' spans are packed into accumulators of their own, since each
// accumulator handed over costs about 1 us; the one slot of a tile whose tokens
// all have that adapter goes straight into the shared product's.
//
// The sum over the reduction is kept in FP32 as FP32 should be: the tensor
// cores' own accumulation loses about 2^-24 of the running sum at each MMA,
// always towards zero, which grows with the length.  Here a tensor-memory
// accumulator takes promote_kblocks k-blocks and the epilogue warps add it, rounded to
// nearest, to sums they hold in registers, while the MMAs fill the other accumulator.
//
// Up to 128 tokens (one token tile, bound by the read of W) there is time to spare
// on the epilogue warps and none in the handing over of accumulators, each about
// 1 us: there the warps form u B_a themselves, FP32 on the CUDA cores, while the
// shared product is under way.  A lane holds its row of the adapter, fetched ahead
// with cp.async, and goes over that adapter's tokens; the results wait in spare
// tensor-memory columns, which, unlike registers, can be addressed by a token
// number, until they are added to the sums.
//
// Roles, ring, tile order, TMA epilogue and the unwinding after a timeout are
// those of gemm_tc.cuh.
#pragma once
#include "gemm_tc.cuh"

namespace lmh {

// k-blocks of 64 per tensor-memory accumulation.  FP32 logits: 12 (768 terms) keep
// the error of a product at 7.1e-7 of its norm at any length (8: 4.7e-7, 16:
// 1.0e-6, one accumulation of 4096 terms: 4.4e-6, of 32768: 3.8e-5; an FP32 product
// on the CUDA cores: 6.1e-7 at 4096).  A switch of accumulators costs the tensor
// pipe about 0.2 us: 4096 x 4096 x 128256 takes 3163, 3101, 3043 us with 8, 12, 16
// and 2966 without.  FP32 dX: 8, because dlogits has one large term per row, the
// target's, after which every MMA loses its share of the whole sum (9.8e-7 with
// 12); the logits of up to 64 tokens: 8 too, since they wait for W and lose nothing by
// it.  BF16 outputs round at 2e-3, so 64 (4e-6) do; BF16 logits whose tiles are cut along
// K are summed in FP32 scratch, and as FP32 logits are.
__host__ __device__ constexpr int promote_kblocks(int out_bytes, bool gradient, int bn)
{
    return out_bytes == 4 ? (gradient || bn <= 64 ? 8 : 12) : 64;
}

constexpr int kSlotMaskWords = 8;  // one bit per token of a tile of up to 256

// A slot in the table: its adapter, and where its span lies among the tile's
// tokens (lo, span: multiples of 32) and in its accumulator (off).
__host__ __device__ constexpr int32_t slot_info(int lo, int span, int off, int last)
{
    return lo / 32 | span / 32 << 4 | off / 32 << 8 | last << 12;
}
__host__ __device__ constexpr int slot_lo(int32_t i) { return (i & 15) * 32; }
__host__ __device__ constexpr int slot_span(int32_t i) { return (i >> 4 & 15) * 32; }
__host__ __device__ constexpr int slot_off(int32_t i) { return (i >> 8 & 15) * 32; }
__host__ __device__ constexpr bool slot_last(int32_t i) { return i >> 12 & 1; }  // of its accumulator

// What a tile split into `parts` puts into scratch: the parts, and the adapters' term
// where it is formed by itself.
__host__ __device__ constexpr int split_slabs(int bn, int parts) { return parts + (bn <= 128 ? 1 : 0); }

constexpr int kSplitParts = 3;  // BF16 parts of u

// Ring stages (64 columns of the split u) of one slot: up to 16 ranks
// {part 0, 1, 2, zeros} of 16 columns in one; up to 32 {part 0, 1} and {part 2, zeros}
// of 32; above that a stage per part and 64 ranks.
__host__ __device__ constexpr int lora_stages(int rank)
{
    return rank > 32 ? kSplitParts * ((rank + 63) / 64) : rank <= 16 ? 1 : 2;
}

struct LoraParams {
    const int2 *count;         // per token tile: {slots, accumulators they take; 0: the shared one}
    const int2 *slot;          // [token tile][slot_stride]: {adapter, slot_info}
    const uint32_t *slot_mask; // [token tile][max_slots][kSlotMaskWords]: their tokens
    int32_t slot_stride;       // even
    int32_t max_slots;
    int32_t stages_per_slot;   // ring stages of one slot: see lora_stages
    int32_t rank;
    int32_t split_parts;       // parts every tile's reduction is cut into (0: whole tiles)
    int32_t part_kb;           // k-blocks of such a part (the last may have fewer)
    float *scratch;            // [tile][split_slabs][BN][tile's rows]
    const __nv_bfloat16 *adapters;  // [adapter][Mdim][rank], A_MN: [adapter][rank][Mdim]
    const float *t;                 // u (g): [Ndim][rank]
};

// Epilogue warps: sums of a whole tile stay in their registers, 128 per thread
// with a 256-wide tile and eight warps, at most 64 with the narrower ones.
constexpr int lora_epi_warps(int bn) { return bn >= 128 ? 8 : 4; }

// Tensor-memory columns: two accumulators and, up to 128 tokens, the adapters' term.
__host__ __device__ constexpr uint32_t lora_tmem_cols(int bn)
{
    const int want = bn <= 128 ? 3 * bn : 2 * bn;
    uint32_t n = 32;
    while (static_cast<int>(n) < want)
        n *= 2;
    return n;
}

// SPLIT: tiles may be split along the reduction (logits: all are, and the parts go to
// lora_join_kernel).  A parameter of its own, so that the logits' kernels without it
// keep their registers.
template <int BN, bool A_MN, typename OutT, bool TMA_STORE, bool PAIR, int RES = 1, int EW = lora_epi_warps(BN),
          bool SPLIT = A_MN>
__global__ void __launch_bounds__(64 + 32 * EW, RES)
    lora_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmS,
                     const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmP,
                     const GemmParams p, const LoraParams q)
{
    using C = GemmCfg<BN, A_MN, false, PAIR, RES, EW>;
    constexpr int S = C::STAGES;
    // the epilogue warps form the adapters' term; otherwise the tensor cores
    constexpr bool IN_REGS = BN <= 128;
    constexpr uint32_t TMEM_COLS = lora_tmem_cols(BN);
    static_assert(RES * TMEM_COLS <= 512, "tensor memory of the resident CTAs");
    constexpr int kPromote = promote_kblocks(sizeof(OutT), A_MN, BN);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *tiles = smem;
    uint8_t *epi_smem = smem + S * C::STAGE_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + C::EPI_BYTES);
    uint64_t *full = bars;
    uint64_t *empty = bars + S;
    uint64_t *acc_full = bars + 2 * S;
    uint64_t *acc_empty = bars + 2 * S + 2;
    uint64_t *drain = bars + 2 * S + 4;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile uint32_t *issued_sh = tmem_slot + 2;  // k-blocks whose copies this CTA issued

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int unit = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
    const int num_units = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
    const int num_tiles = p.num_m_tiles * p.num_n_tiles;
    const int num_kb = (p.Kdim + kBlockK - 1) / kBlockK;
    // Split along the reduction, the parts go to scratch (tmP) in FP32, where
    // lora_join_kernel adds them; the last part takes the slots.
    // - Fewer tiles than units (few tokens; a narrow model, a small vocabulary): every
    //   tile into split_parts parts, so that most units have one.  Where the epilogue warps form
    //   the adapters' term, each part takes that of its share of the tokens, and it
    //   goes to scratch as one part more: a token's sums are the same wherever in the
    //   batch it stands.
    // - Several waves of dX's tiles: the tiles of a last wave that would leave many units idle in
    //   two, as in gemm_tc_kernel: long part [0, split_kb) on the unit that would have
    //   run the tile, short part on an idle one.
    const bool all_split = SPLIT && q.split_parts > 0;
    const int split_first = !SPLIT ? num_tiles : all_split ? 0 : num_tiles - p.split_tiles;
    constexpr bool ROTATE = !A_MN && BN > 128 && !SPLIT;  // logits of several token tiles
    const int waves = (num_tiles + num_units - 1) / num_units;
    const int num_items = ROTATE ? waves * num_units
                          : all_split ? num_tiles * q.split_parts
                          : p.split_tiles > 0 ? split_first + num_units * p.split_rounds : num_tiles;
    // item -> tile and k-blocks: -1 a whole tile, from 0 on a part, -2 nothing to do
    // ROTATE: the units that share a panel of W have to stay in step for L2 to serve
    // all but one of them, while tiles take longer the more adapters their tokens
    // have.  Each wave starts one tile further on, so that every unit comes by every
    // token tile in turn (with 74 units and 16 token tiles, it would only see those
    // of one parity: 4096 x 4096 x 128256 with 8 adapters read 4.2 GB from DRAM instead
    // of 2.2 and took 3.45 ms instead of 3.28).  The last wave's tiles, fewer than the
    // units, go to the first ones: the last ones start late, where the row kernel ran
    // (200 x 2048 x 60000: 98 against 89 us).  With one narrow token tile there is nothing
    // to gain, and the index arithmetic costs (64 x 4096 x 32768, rank 64: 121 against 107 us).
    auto item_of = [&](int it, int &t, int &kb0, int &kb1) -> int {
        t = it;
        kb0 = 0;
        kb1 = num_kb;
        if (ROTATE) {
            const int w = it / num_units, u = it - w * num_units;
            t = w * num_units + (w + 1 < waves ? (u + w) % num_units : u);
            return t < num_tiles ? -1 : -2;
        }
        if (all_split) {
            t = it / q.split_parts;
            kb0 = (it - t * q.split_parts) * q.part_kb;
            kb1 = min(num_kb, kb0 + q.part_kb);
            return it - t * q.split_parts;
        }
        if (!SPLIT || it < split_first)
            return -1;
        const int j = it - split_first, r = j / num_units, u = j - r * num_units;
        if (u < p.split_tiles) {
            t = split_first + u;
            kb1 = p.split_kb;
            return r == 0 ? 0 : -2;
        }
        const int idx = (u - p.split_tiles) + r * (num_units - p.split_tiles);
        t = split_first + idx;
        kb0 = p.split_kb;
        return idx < p.split_tiles ? 1 : -2;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], EW * C::CTAS);  // one arrival per epilogue warp
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        *issued_sh = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        if (!IN_REGS) {
            tma_prefetch_desc(&tmS);
            tma_prefetch_desc(&tmU);
        }
        if (TMA_STORE)
            tma_prefetch_desc(&tmC);
        if (all_split || (SPLIT && p.split_tiles > 0))
            tma_prefetch_desc(&tmP);
    }
    if (warp == 1) {
        if (PAIR)
            tmem_alloc_pair(tmem_slot, TMEM_COLS);
        else
            tmem_alloc(tmem_slot, TMEM_COLS);
    }
    tc_fence_before();
    if (PAIR)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // X, W and dlogits were complete before the row kernel of this call began, and
    // this kernel starts once the expand kernel after it has: only what those two
    // write (u, the slots) has to be waited for, by each role that reads it.
    pdl_launch_dependents();

    const uint64_t pol_a = policy_of(p.l2_a);
    const uint64_t pol_b = policy_of(p.l2_b);
    const uint64_t pol_n = policy_of(0);
    // Arms the full barrier of ring slot `stage` (the leader's, which counts the
    // bytes of both CTAs) and returns where this CTA's copies signal it.  Every
    // stage, of the shared product or of a slot, has STAGE_BYTES per CTA.
    auto arm = [&](uint32_t stage) -> uint32_t {
        if (leader)
            mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES * C::CTAS);
        return PAIR ? mapa_shared(smem_u32(&full[stage]), 0) : 0u;
    };
    auto load2 = [&](const CUtensorMap *m, uint32_t stage, uint32_t fb, void *dst, int c0, int c1, uint64_t pol) {
        if (PAIR)
            tma_load_2d_pair(m, fb, dst, c0, c1, pol);
        else
            tma_load_2d(m, &full[stage], dst, c0, c1, pol);
    };
    auto load3 = [&](const CUtensorMap *m, uint32_t stage, uint32_t fb, void *dst, int c0, int c1, int c2) {
        if (PAIR)
            tma_load_3d_pair(m, fb, dst, c0, c1, c2, pol_n);
        else
            tma_load_3d(m, &full[stage], dst, c0, c1, c2, pol_n);
    };
    auto issue_kblock = [&](uint32_t stage, int m0, int nb0, int k0) {
        uint8_t *sa = tiles + stage * C::STAGE_BYTES;
        const uint32_t fb = arm(stage);
        if (A_MN) {
#pragma unroll
            for (int j = 0; j < kBlockM / 64; ++j)
                load2(&tmA, stage, fb, sa + j * 64 * kBlockK * 2, m0 + 64 * j, k0, pol_a);
        } else {
            load2(&tmA, stage, fb, sa, k0, m0, pol_a);
        }
        load2(&tmB, stage, fb, sa + C::A_BYTES, k0, nb0, pol_b);
    };
    // One ring stage of an adapter: its 64 ranks from r0 against the rows m0.. of
    // the output (ranks past the last read as zero), and BN_CTA rows of the
    // split u from row urow.
    auto issue_slot = [&](uint32_t stage, int m0, int id, int r0, int urow) {
        uint8_t *sa = tiles + stage * C::STAGE_BYTES;
        const uint32_t fb = arm(stage);
        if (A_MN) {
#pragma unroll
            for (int j = 0; j < kBlockM / 64; ++j)
                load3(&tmS, stage, fb, sa + j * 64 * kBlockK * 2, m0 + 64 * j, r0, id);
        } else {
            load3(&tmS, stage, fb, sa, r0, m0, id);
        }
        load2(&tmU, stage, fb, sa + C::A_BYTES, 0, urow, pol_n);
    };
    const int sps = q.stages_per_slot;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            uint32_t issued = 0;
            bool ok = true;
            bool slots_there = false;
            for (int it = unit; it < num_items && ok; it += num_units) {
                int t, kb0, kb1, mt, nt;
                if (item_of(it, t, kb0, kb1) == -2)
                    continue;
                tile_coords(t, p, mt, nt);
                const int m0 = mt * C::TILE_M + static_cast<int>(rank) * kBlockM;
                const int nb0 = nt * BN + static_cast<int>(rank) * C::BN_CTA;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    issue_kblock(stage, m0, nb0, kb * kBlockK);
                    ++issued;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (IN_REGS || kb1 != num_kb)
                    continue;
                if (!slots_there)
                    pdl_wait();
                slots_there = true;
                const int ns = q.count[nt].x;
                const int4 *two = reinterpret_cast<const int4 *>(q.slot + static_cast<int64_t>(nt) * q.slot_stride);
                for (int s2 = 0; s2 < ns && ok; s2 += 2) {
                    const int4 e = two[s2 >> 1];
#pragma unroll 1
                    for (int s = s2; s < s2 + 2 && s < ns && ok; ++s) {
                        const int id = s & 1 ? e.z : e.x, info = s & 1 ? e.w : e.y;
                        const int row = slot_lo(info) + static_cast<int>(rank) * (slot_span(info) / C::CTAS);
#pragma unroll 1
                        for (int j = 0; j < sps; ++j) {
                            if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.wait_limit_ns)) {
                                ok = false;
                                break;
                            }
                            issue_slot(stage, m0, id, j / kSplitParts * 64, (nt * sps + j) * BN + row);
                            ++issued;
                            if (++stage == S) {
                                stage = 0;
                                phase ^= 1;
                            }
                        }
                    }
                }
            }
            *issued_sh = issued;
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (pair: leader only)
        if (lane == 0 && leader) {
            uint32_t stage = 0, phase = 0;
            uint32_t acc = 0, acc_phase = 0;
            bool ok = true;
            bool slots_there = false;
            // a stage whose copies have landed, its descriptors' bases
            uint32_t sa = 0, sb = 0, d_tmem = 0;
            uint32_t idesc = C::IDESC;
            auto mma = [&](int ka, int kbb, uint32_t accumulate) {
                // K-major: 32 bytes along the swizzled row per 16 of the
                // reduction.  MN-major: 16 rows of 128 bytes.
                const uint64_t da = A_MN ? smem_desc_sw128(sa + ka * 2048, 64 * kBlockK * 2, 1024)
                                         : smem_desc_sw128(sa + ka * 32, 16, 1024);
                const uint64_t db = smem_desc_sw128(sb + kbb * 32, 16, 1024);
                if (PAIR)
                    mma_bf16_pair(d_tmem, da, db, idesc, accumulate);
                else
                    mma_bf16(d_tmem, da, db, idesc, accumulate);
            };
            auto begin_acc = [&]() -> bool {
                if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1, abort_flag, p.wait_limit_ns))
                    return false;
                tc_fence_after();
                d_tmem = tmem_base + acc * BN;
                return true;
            };
            auto end_acc = [&]() {
                if (PAIR)
                    mma_commit_pair(&acc_full[acc], 0x3);
                else
                    mma_commit(&acc_full[acc]);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            };
            auto begin_stage = [&]() -> bool {
                if (!mbar_wait(&full[stage], phase, abort_flag, p.wait_limit_ns))
                    return false;
                tc_fence_after();
                sa = smem_u32(tiles + stage * C::STAGE_BYTES);
                sb = sa + C::A_BYTES;
                return true;
            };
            auto end_stage = [&]() {
                // frees the smem slot (of both CTAs) when these MMAs finish
                if (PAIR)
                    mma_commit_pair(&empty[stage], 0x3);
                else
                    mma_commit(&empty[stage]);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            };
            for (int it = unit; it < num_items && ok; it += num_units) {
                int t, kb_first, kb_end, mt, nt;
                if (item_of(it, t, kb_first, kb_end) == -2)
                    continue;
                tile_coords(t, p, mt, nt);
                const bool slots = !IN_REGS && kb_end == num_kb;
                // slots, their accumulators and the first two slots, wanted after the
                // shared product
                int2 n = {0, 0};
                int4 two = {0, 0, 0, 0};
                const int4 *table = reinterpret_cast<const int4 *>(q.slot + static_cast<int64_t>(nt) * q.slot_stride);
                if (slots && slots_there) {
                    n = q.count[nt];
                    two = table[0];
                }
                idesc = C::IDESC;
                for (int kb0 = kb_first; kb0 < kb_end && ok; kb0 += kPromote) {
                    if (!begin_acc()) {
                        ok = false;
                        break;
                    }
                    const int kb1 = min(kb_end, kb0 + kPromote);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!begin_stage()) {
                            ok = false;
                            break;
                        }
#pragma unroll
                        for (int k = 0; k < kBlockK / kUmmaK; ++k)
                            mma(k, k, (kb != kb0 || k != 0) ? 1u : 0u);
                        end_stage();
                    }
                    if (slots && kb1 == kb_end && !slots_there) {
                        pdl_wait();
                        slots_there = true;
                        n = q.count[nt];
                        two = table[0];
                    }
                    // a slot that takes no accumulator of its own stays with this one
                    if (ok && !(kb1 == kb_end && n.x > 0 && n.y == 0))
                        end_acc();
                }
                bool open = n.x > 0 && n.y == 0;  // whether the current accumulator is begun
                const uint32_t joined = open ? 1u : 0u;
#pragma unroll 1
                for (int s = 0; s < n.x && ok; ++s) {
                    if (s > 0 && (s & 1) == 0)
                        two = table[s >> 1];
                    const int info = s & 1 ? two.w : two.y;
                    if (!open && !begin_acc()) {
                        ok = false;
                        break;
                    }
                    open = !slot_last(info);
                    d_tmem = tmem_base + acc * BN + slot_off(info);
                    idesc = (C::IDESC & ~(0x3fu << 17)) | (static_cast<uint32_t>(slot_span(info)) >> 3) << 17;
#pragma unroll 1
                    for (int j = 0; j < sps; ++j) {
                        if (!begin_stage()) {
                            ok = false;
                            break;
                        }
                        if (q.rank <= 16) {
                            mma(0, 0, joined);
                            mma(0, 1, 1u);
                            mma(0, 2, 1u);
                        } else if (q.rank <= 32) {
                            mma(0, 0, j != 0 ? 1u : joined);
                            mma(1, 1, 1u);
                            if (j == 0) {
                                mma(0, 2, 1u);
                                mma(1, 3, 1u);
                            }
                        } else {
                            // 64 ranks: one part after the other
                            const int steps = min(4, (q.rank - j / kSplitParts * 64 + kUmmaK - 1) / kUmmaK);
                            for (int k = 0; k < steps; ++k)
                                mma(k, k, (j != 0 || k != 0) ? 1u : joined);
                        }
                        end_stage();
                    }
                    if (ok && !open)
                        end_acc();
                }
            }
            // wait until every MMA issued by this thread has completed
            if (PAIR)
                mma_commit_pair(drain, 0x1);
            else
                mma_commit(drain);
            volatile int no_abort = 0;
            mbar_wait(drain, 0, &no_abort, kDrainLimitNs);
        }
    } else {
        // ------------------------------------------------ epilogue (warps 2 .. 2 + EW - 1)
        constexpr int CH = C::EPI_CHUNK;
        constexpr int COLS = BN / (EW / 4);  // columns this warp's quarter and half hold
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;
        OutT *out = static_cast<OutT *>(p.out);
        const uint64_t pol_out = policy_of(p.l2_out);
        OutT *slots = reinterpret_cast<OutT *>(epi_smem + (warp - 2) * C::NSLOT * C::EPI_SLOT_BYTES);
        constexpr int SLOT_ELEMS = C::EPI_SLOT_BYTES / static_cast<int>(sizeof(float));
        uint32_t slot = 0;
        const uint32_t empty_addr0 = PAIR ? mapa_shared(smem_u32(&acc_empty[0]), 0) : 0u;
        uint32_t acc = 0, acc_phase = 0;
        bool ok = true;
        pdl_wait();
        for (int it = unit; it < num_items && ok; it += num_units) {
            int t, kb0, kb1, mt, nt;
            const int part = item_of(it, t, kb0, kb1);
            if (part == -2)
                continue;
            tile_coords(t, p, mt, nt);
            const int mbase = mt * C::TILE_M + static_cast<int>(rank) * kBlockM;
            const int m = mbase + quarter * 32 + lane;
            const int n0 = nt * BN + half * COLS;
            const int chunks = (kb1 - kb0 + kPromote - 1) / kPromote;
            const int2 n = kb1 == num_kb || (IN_REGS && all_split) ? q.count[nt] : make_int2(0, 0);
            const int ns = n.x;
            const int all = IN_REGS ? chunks : chunks + n.y;
            const int2 *table = q.slot + static_cast<int64_t>(nt) * q.slot_stride;
            // this warp's columns of the tile's slot masks, one slot ahead
            const uint32_t *masks = q.slot_mask + static_cast<int64_t>(nt) * q.max_slots * kSlotMaskWords +
                                    half * COLS / 32;
            constexpr int MW = COLS < 32 ? 1 : COLS / 32;
            float sum[COLS];
#pragma unroll
            for (int i = 0; i < COLS; ++i)
                sum[i] = 0.f;
            int ch = 0;
            // adds the accumulator that has come full to the sums and frees it
            auto take_shared = [&]() {
                tc_fence_after();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN + half * COLS;
#pragma unroll
                for (int c = 0; c < COLS; c += 16) {
                    uint32_t r[32];
                    tmem_ld_chunk<16>(taddr + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        sum[c + j] += __uint_as_float(r[j]);
                }
            };
            auto release_acc = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR)
                        mbar_arrive_cluster(empty_addr0 + acc * 8);
                    else
                        mbar_arrive(&acc_empty[acc]);
                }
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1;
                }
                ++ch;
            };
            // where the adapters' term waits, and the tokens that have one
            const uint32_t stash = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 2 * BN + half * COLS;
            uint32_t has[MW] = {}, own[MW];  // (of this part's tokens)
            if constexpr (IN_REGS) {
                // A piece is 8 ranks of one slot: 16 bytes per lane, its row of the
                // adapter, through the lane's own places in the staging slots (free
                // until the tile's stores), up to AHEAD pieces before they are used.
                constexpr int ROOM = C::NSLOT * C::EPI_SLOT_BYTES / 512;
                constexpr int AHEAD = ROOM < 16 ? ROOM : 16;
                constexpr int RC = 32;  // ranks held in registers at once
                uint4 *ring = reinterpret_cast<uint4 *>(slots);
                const int per_slot = q.rank / 8;
                const int pieces = ns * per_slot;
                const bool in = m < p.Mdim;
#pragma unroll
                for (int i = 0; i < MW; ++i)
                    own[i] = 0xffffffffu;
                if (all_split) {  // every split_parts-th token
#pragma unroll
                    for (int i = 0; i < MW; ++i) {
                        const int c = i * 32 + lane;
                        own[i] = __ballot_sync(0xffffffffu, c < COLS && (half * COLS + c) % q.split_parts == part);
                    }
                }
                int fs = 0, fr = 0, fetched = 0;  // slot and rank block of the next fetch
                if (lane == 0)
                    bulk_wait_read<0>();  // the last tile's stores have left the slots
                __syncwarp();
                auto fetch = [&]() {
                    if (fetched < pieces) {
                        const __nv_bfloat16 *src =
                            q.adapters + (static_cast<int64_t>(table[fs].x) * p.Mdim + (in ? m : 0)) * q.rank + fr * 8;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                         smem_u32(ring + (fetched % AHEAD) * 32 + lane)),
                                     "l"(src), "r"(in ? 16 : 0)
                                     : "memory");
                        ++fetched;
                        if (++fr == per_slot) {
                            fr = 0;
                            ++fs;
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                constexpr bool RING = !A_MN && !SPLIT;  // a part has few slots
                if constexpr (RING)
                    for (int i = 0; i < AHEAD - 1; ++i)
                        fetch();
                int used = 0;
#pragma unroll 1
                for (int s = 0; s < ns; ++s) {
                    // an accumulator that is full meanwhile is not kept waiting
                    if (ch < chunks &&
                        __all_sync(0xffffffffu, mbar_test_wait(smem_u32(&acc_full[acc]), acc_phase))) {
                        take_shared();
                        release_acc();
                    }
                    uint32_t mask[MW], any = 0;
#pragma unroll
                    for (int i = 0; i < MW; ++i) {
                        mask[i] = masks[s * kSlotMaskWords + i] & own[i];
                        has[i] |= mask[i];
                        any |= mask[i];
                    }
                    if (SPLIT && any == 0)
                        continue;
#pragma unroll 1
                    for (int r0 = 0; r0 < q.rank; r0 += RC) {
                        const int n8 = min(RC / 8, (q.rank - r0) / 8);
                        float b[RC];
#pragma unroll
                        for (int k = 0; k < RC / 8; ++k) {
                            if (k >= n8)
                                continue;
                            if constexpr (!A_MN) {
                                uint4 v = make_uint4(0, 0, 0, 0);
                                if constexpr (RING) {
                                    asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 2) : "memory");
                                    v = ring[(used++ % AHEAD) * 32 + lane];
                                    fetch();
                                } else if (in) {
                                    v = *reinterpret_cast<const uint4 *>(
                                        q.adapters + (static_cast<int64_t>(table[s].x) * p.Mdim + m) * q.rank + r0 + 8 * k);
                                }
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    b[8 * k + 2 * j] = __uint_as_float(w[j] << 16);
                                    b[8 * k + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                                }
                            } else {
                                const __nv_bfloat16 *src =
                                    q.adapters + (static_cast<int64_t>(table[s].x) * q.rank + r0 + 8 * k) * p.Mdim + (in ? m : 0);
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    b[8 * k + j] = in ? __bfloat162float(src[static_cast<int64_t>(j) * p.Mdim]) : 0.f;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < MW; ++i) {
#pragma unroll 1
                            for (uint32_t left = mask[i]; left; left &= left - 1) {
                                const int c = i * 32 + __ffs(left) - 1;
                                const float4 *tp = reinterpret_cast<const float4 *>(
                                    q.t + static_cast<int64_t>(n0 + c) * q.rank + r0);
                                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                for (int k = 0; k < RC / 4; ++k) {
                                    if (k >= 2 * n8)
                                        continue;
                                    const float4 x = tp[k];
                                    d[0] = fmaf(x.x, b[4 * k], d[0]);
                                    d[1] = fmaf(x.y, b[4 * k + 1], d[1]);
                                    d[2] = fmaf(x.z, b[4 * k + 2], d[2]);
                                    d[3] = fmaf(x.w, b[4 * k + 3], d[3]);
                                }
                                float sum4 = (d[0] + d[1]) + (d[2] + d[3]);
                                if (r0 > 0) {
                                    tmem_st_wait();
                                    const uint32_t before = tmem_ld1(stash + c);
                                    tmem_ld_wait();
                                    sum4 += __uint_as_float(before);
                                }
                                tmem_st1(stash + c, __float_as_uint(sum4));
                            }
                        }
                    }
                }
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                tmem_st_wait();
                __syncwarp();
            }
            int s = 0;  // the next slot to be added, its place and tokens fetched ahead
            int32_t info = 0;
            uint32_t mask[MW] = {};
            auto fetch_slot = [&]() {
                if (s < ns) {
                    info = table[s].y;
#pragma unroll
                    for (int i = 0; i < MW; ++i)
                        mask[i] = masks[s * kSlotMaskWords + i];
                }
            };
            if (!IN_REGS && n.y > 0)
                fetch_slot();
#pragma unroll 1
            while (ch < all) {
                const bool shared = IN_REGS || ch < chunks;
                // every lane waits, then the warp agrees, so the .sync.aligned
                // tensor-memory loads below always run with the full warp
                const bool got = mbar_wait(&acc_full[acc], acc_phase, abort_flag, p.wait_limit_ns);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                if (shared) {
                    take_shared();
                } else {
                    tc_fence_after();
                    bool last;
                    do {
                        last = slot_last(info);
                        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN +
                                               half * COLS + slot_off(info) - slot_lo(info);
                        uint32_t now[MW];
#pragma unroll
                        for (int i = 0; i < MW; ++i)
                            now[i] = mask[i];
                        ++s;
                        fetch_slot();
#pragma unroll
                        for (int c = 0; c < COLS; c += 16) {
                            const uint32_t m16 = (now[c / 32] >> (c & 31)) & 0xffffu;
                            if (m16 == 0)
                                continue;
                            uint32_t r[32];
                            tmem_ld_chunk<16>(taddr + c, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (m16 >> j & 1u)
                                    sum[c + j] += __uint_as_float(r[j]);
                        }
                    } while (!last);
                }
                release_acc();
            }
            if (!ok)
                break;
            if (IN_REGS && all_split) {
                float *slab = q.scratch + quarter * 32 + lane +
                              (static_cast<int64_t>(t * split_slabs(BN, q.split_parts) + q.split_parts) * BN + half * COLS) *
                                  C::TILE_M;
#pragma unroll
                for (int c = 0; c < COLS; c += 16) {
                    const uint32_t o16 = (own[c / 32] >> (c & 31)) & 0xffffu;
                    const uint32_t m16 = (has[c / 32] >> (c & 31)) & 0xffffu;
                    if (o16 == 0)
                        continue;
                    uint32_t r[32];
                    tmem_ld_chunk<16>(stash + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (o16 >> j & 1u)
                            slab[(c + j) * C::TILE_M] = m16 >> j & 1u ? __uint_as_float(r[j]) : 0.f;
                }
            } else if constexpr (IN_REGS) {
                // last, whenever the accumulators came, so that the order is always the same
#pragma unroll
                for (int c = 0; c < COLS; c += 16) {
                    const uint32_t m16 = (has[c / 32] >> (c & 31)) & 0xffffu;
                    if (m16 == 0)
                        continue;
                    uint32_t r[32];
                    tmem_ld_chunk<16>(stash + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (m16 >> j & 1u)
                            sum[c + j] += __uint_as_float(r[j]);
                }
            }
            if (SPLIT && part >= 0) {
                const int slabs = all_split ? split_slabs(BN, q.split_parts) : 2;
                const int y = ((t - split_first) * slabs + part) * BN + half * COLS;  // scratch row
                float *fslots = reinterpret_cast<float *>(slots);
#pragma unroll
                for (int c = 0; c < COLS; c += CH) {
                    if (n0 + c < p.Ndim) {
                        if (lane == 0)
                            bulk_wait_read<C::NSLOT - 1>();
                        __syncwarp();
                        float *buf = fslots + slot * (C::EPI_SLOT_BYTES / 4);
#pragma unroll
                        for (int j = 0; j < CH; ++j)
                            buf[j * 32 + lane] = sum[c + j];
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&tmP, buf, static_cast<int>(rank) * kBlockM + quarter * 32, y + c);
                            bulk_commit();
                        }
                        slot = slot + 1 == C::NSLOT ? 0 : slot + 1;
                    }
                }
                continue;
            }
#pragma unroll
            for (int c = 0; c < COLS; c += CH) {
                if (TMA_STORE) {
                    if (n0 + c < p.Ndim) {
                        // the slot is free once the store issued NSLOT sub-tiles
                        // ago has finished reading it
                        if (lane == 0)
                            bulk_wait_read<C::NSLOT - 1>();
                        __syncwarp();
                        OutT *buf = slots + slot * SLOT_ELEMS;
#pragma unroll
                        for (int j = 0; j < CH; ++j)
                            stage_out(buf + j * 32 + lane, __float_as_uint(sum[c + j]));
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (p.l2_out)
                                tma_store_2d_hint(&tmC, buf, mbase + quarter * 32, n0 + c, pol_out);
                            else
                                tma_store_2d(&tmC, buf, mbase + quarter * 32, n0 + c);
                            bulk_commit();
                        }
                        slot = slot + 1 == C::NSLOT ? 0 : slot + 1;
                    }
                } else if (m < p.Mdim) {
                    OutT *o = out + static_cast<int64_t>(n0 + c) * p.ldo + m;
#pragma unroll
                    for (int j = 0; j < CH; ++j)
                        if (n0 + c + j < p.Ndim)
                            store_out(o + static_cast<int64_t>(j) * p.ldo, __float_as_uint(sum[c + j]));
                }
            }
        }
        if (TMA_STORE && lane == 0)
            bulk_wait_all();  // every output byte written before the CTA exits
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) {
        // as in gemm_tc_kernel: after a timeout the CTA that is behind issues the
        // k-blocks it missed (any data: the stages are of one size), so that
        // every phase a copy belongs to completes before either CTA leaves
        cluster_sync();
        const uint32_t peer = rank ^ 1u;
        const int peer_abort = static_cast<int>(
            ld_shared_cluster_u32(mapa_shared(smem_u32(const_cast<int *>(abort_flag)), peer)));
        if (*abort_flag || peer_abort) {
            if (threadIdx.x == 0) {
                const uint32_t mine = *issued_sh;
                const uint32_t theirs = ld_shared_cluster_u32(
                    mapa_shared(smem_u32(const_cast<uint32_t *>(issued_sh)), peer));
                const uint32_t all = mine > theirs ? mine : theirs;
                for (uint32_t i = mine; i < all; ++i)
                    issue_kblock(i % S, static_cast<int>(rank) * kBlockM,
                                 static_cast<int>(rank) * C::BN_CTA, 0);
                if (leader) {
                    volatile int no_abort = 0;
                    for (uint32_t i = all > S ? all - S : 0; i < all; ++i)
                        mbar_wait(&full[i % S], (i / S) & 1u, &no_abort, kDrainLimitNs);
                }
            }
            cluster_sync();
        }
        cluster_sync();
    } else {
        if (*abort_flag && threadIdx.x == 0) {
            const uint32_t all = *issued_sh;
            volatile int no_abort = 0;
            for (uint32_t i = all > S ? all - S : 0; i < all; ++i)
                mbar_wait(&full[i % S], (i / S) & 1u, &no_abort, kDrainLimitNs);
        }
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if (PAIR)
            tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else
            tmem_dealloc(tmem_base, TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag && p.status)
        atomicOr(p.status, 2);
}

// out = the parts of the split tiles added in order.  grid (split tiles, row groups).
// scratch [tile][part][bn][tile_m].
constexpr int kJoinRows = 8;

template <typename OutT>
__global__ void __launch_bounds__(256)
    lora_join_kernel(const float *__restrict__ scratch, OutT *__restrict__ out, const GemmParams p, int32_t split_first,
                     int32_t parts, int32_t bn, int32_t tile_m)
{
    pdl_wait();
    pdl_launch_dependents();
    int mt, nt;
    tile_coords(split_first + static_cast<int>(blockIdx.x), p, mt, nt);
    const int lanes = tile_m / 4, c = static_cast<int>(threadIdx.x) % lanes * 4;
    const int m = mt * tile_m + c;
    if (m >= p.Mdim)
        return;
    for (int r = threadIdx.x / lanes; r < kJoinRows; r += 256 / lanes) {
        const int row = blockIdx.y * kJoinRows + r;
        const int64_t n = static_cast<int64_t>(nt) * bn + row;
        if (n >= p.Ndim)
            return;
        const float *s = scratch + (static_cast<int64_t>(blockIdx.x) * parts * bn + row) * tile_m + c;
        float4 a = *reinterpret_cast<const float4 *>(s);
#pragma unroll 8
        for (int k = 1; k < parts; ++k) {
            const float4 b = *reinterpret_cast<const float4 *>(s + static_cast<int64_t>(k) * bn * tile_m);
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
        }
        OutT *o = out + n * p.ldo + m;
        const float v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (m + j < p.Mdim)
                store_out(o + j, __float_as_uint(v[j]));
    }
}

}  // namespace lmh
