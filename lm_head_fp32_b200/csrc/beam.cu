// beam.cu -- C ABI of the beam-search calls (declared in include/lmhead.h):
// argument validation and launches of beam_kernels.cuh.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "lmhead.h"
#include "beam_kernels.cuh"
#include "host.cuh"

namespace {

using namespace lmh::host;

// How a row is cut into parts of `batches` batches, one CTA each: enough parts
// that the CTAs fill the GPU (twice as many: 64 x 8 x 151936 75.5 against 72.6 us,
// 16 x 4 x 128256 22.2 against 17.8), and no more, since each part hands
// C candidates on.
struct BeamParts {
    int64_t batches, parts;
};
constexpr int64_t kBeamCtas = 148 * 6;  // CTAs aimed at: what the SMs hold at once
BeamParts beam_parts(int64_t rows, int64_t V)
{
    const int64_t per_row = (V + lmh::kBeamBatch - 1) / lmh::kBeamBatch;  // batches
    int64_t batches = rows * per_row / kBeamCtas;
    batches = batches > lmh::kBeamMaxBatches ? lmh::kBeamMaxBatches : batches;
    batches = batches < 1 ? 1 : batches;
    return {batches, (per_row + batches - 1) / batches};
}

bool beam_dims_ok(int64_t N, int64_t W, int64_t V, int64_t C)
{
    if (N < 1 || W < 1 || W > lmh::kBeamMaxWidth || V < 1 || V > kMaxDim || C < 1 ||
        C > lmh::kBeamMaxCand || N > kMaxDim / W)
        return false;
    const int64_t parts = beam_parts(N * W, V).parts;
    // CTAs of the scan, and an entry's candidates in the merge, are counted in 32 bits
    return N * W <= kMaxDim / parts && W * parts <= kMaxDim / C;
}

int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

template <typename T>
lmh_status_t launch_scan(const void *logits, const float *scores, const int32_t *done,
                         lmh::BeamPartial *part, lmh::BeamCand *cand, int64_t N, int64_t W, int64_t V,
                         int64_t C, const BeamParts &bp, int32_t *status, cudaStream_t s)
{
    return launch_ex(lmh::beam_scan_kernel<T>, dim3(static_cast<unsigned>(N * W * bp.parts)),
                     dim3(lmh::kBeamThreads), 0, s, 1u, static_cast<const T *>(logits), scores, done,
                     part, cand, static_cast<int32_t>(W), V, static_cast<int32_t>(C),
                     static_cast<int32_t>(bp.parts), static_cast<int32_t>(bp.batches), status);
}

template <typename VecT, int MAXW>
lmh_status_t launch_reorder(const lmh::ReorderParams &p, int64_t N, int num_states, cudaStream_t s)
{
    constexpr int64_t per_block = lmh::kReorderThreads * lmh::kReorderColumns;
    const int64_t need = (static_cast<int64_t>(p.columns) + per_block - 1) / per_block;
    // several waves of blocks over all entries and states; a thread then takes more columns
    const int64_t cap = (num_sms() * 64 + N * num_states - 1) / (N * num_states);
    const int64_t grid = need < cap ? need : cap;
    return launch_ex(lmh::beam_reorder_kernel<VecT, MAXW>,
                     dim3(static_cast<unsigned>(grid), static_cast<unsigned>(N),
                          static_cast<unsigned>(num_states)),
                     dim3(lmh::kReorderThreads), 0, s, 1u, p);
}

template <typename VecT>
lmh_status_t dispatch_reorder(const lmh::ReorderParams &p, int64_t N, int num_states, cudaStream_t s)
{
    if (p.W <= 4)
        return launch_reorder<VecT, 4>(p, N, num_states, s);
    if (p.W <= 8)
        return launch_reorder<VecT, 8>(p, N, num_states, s);
    if (p.W <= 16)
        return launch_reorder<VecT, 16>(p, N, num_states, s);
    if constexpr (sizeof(VecT) <= 8)
        if (p.W <= 32)
            return launch_reorder<VecT, 32>(p, N, num_states, s);
    if constexpr (sizeof(VecT) <= 4)
        return launch_reorder<VecT, 64>(p, N, num_states, s);
    return LMH_ERR_UNSUPPORTED;
}

// The geometry of a state: dimensions from the smallest stride up, each of which steps
// over all that lies below it (`below` bytes, from the first to the last).
struct Geometry {
    int64_t run = 0;
    int n = 0;
    int64_t extent[5], stride[5], below[5];
};

// Whether two states of this geometry share memory, d bytes apart: whether two elements,
// one of each, come to lie within a run of each other.  In every dimension only the two
// steps next to d can bring them together, since all that lies below moves them by less.
bool states_meet(const Geometry &g, int64_t d, int dim)
{
    if (dim < 0)
        return d > -g.run && d < g.run;
    const int64_t s = g.stride[dim];
    const int64_t q0 = d >= 0 ? d / s : -((-d + s - 1) / s);  // rounded down
    for (int64_t q = q0; q <= q0 + 1; ++q) {
        const int64_t left = d - q * s;
        if (q > -g.extent[dim] && q < g.extent[dim] && left > -g.below[dim] && left < g.below[dim] &&
            states_meet(g, left, dim - 1))
            return true;
    }
    return false;
}

}  // namespace

extern "C" {

int64_t beam_select_workspace_bytes(int64_t N, int64_t W, int64_t V, int64_t C)
{
    if (!beam_dims_ok(N, W, V, C))
        return -1;
    const int64_t parts = N * W * beam_parts(N * W, V).parts;
    return align16(parts * static_cast<int64_t>(sizeof(lmh::BeamPartial))) +
           parts * C * static_cast<int64_t>(sizeof(lmh::BeamCand));
}

lmh_status_t beam_select(const void *logits, int32_t logits_dtype, const float *scores,
                         const int32_t *done, float *cand_score, int32_t *cand_beam,
                         int64_t *cand_token, float *next_score, int32_t *next_beam,
                         int64_t *next_token, void *workspace, int64_t workspace_bytes, int64_t N,
                         int64_t W, int64_t V, int64_t C, int64_t eos, int32_t *status,
                         lmh_stream_t stream)
{
    if (!logits || !scores || !cand_score || !cand_beam || !cand_token || !workspace ||
        !beam_dims_ok(N, W, V, C) || eos < -1 || eos >= V)
        return LMH_ERR_INVALID_ARG;
    const bool next = next_score || next_beam || next_token;
    if (next && (!next_score || !next_beam || !next_token))
        return LMH_ERR_INVALID_ARG;
    // each beam ends at most one candidate, so this many leave W that go on
    if (next && C < (eos < 0 ? W : 2 * W))
        return LMH_ERR_INVALID_ARG;
    if (workspace_bytes < beam_select_workspace_bytes(N, W, V, C))
        return LMH_ERR_INVALID_ARG;
    if (bad_dtype(logits_dtype))
        return LMH_ERR_UNSUPPORTED;
    if (!aligned(logits, logits_dtype == LMH_F32 ? 4 : 2) || !aligned(scores, 4) ||
        !aligned(done, 4) || !aligned(cand_score, 4) || !aligned(cand_beam, 4) ||
        !aligned(cand_token, 8) || !aligned(next_score, 4) || !aligned(next_beam, 4) ||
        !aligned(next_token, 8) || !aligned(workspace, 16))
        return LMH_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const BeamParts bp = beam_parts(N * W, V);
    auto *part = static_cast<lmh::BeamPartial *>(workspace);
    auto *cand = reinterpret_cast<lmh::BeamCand *>(
        static_cast<uint8_t *>(workspace) +
        align16(N * W * bp.parts * static_cast<int64_t>(sizeof(lmh::BeamPartial))));
    const lmh_status_t r =
        logits_dtype == LMH_F32
            ? launch_scan<float>(logits, scores, done, part, cand, N, W, V, C, bp, status, s)
            : launch_scan<__nv_bfloat16>(logits, scores, done, part, cand, N, W, V, C, bp, status, s);
    if (r != LMH_OK)
        return r;
    const lmh::BeamOut o{cand_score, cand_beam, cand_token, next_score, next_beam, next_token};
    return launch_ex(lmh::beam_merge_kernel, dim3(static_cast<unsigned>(N)), dim3(lmh::kBeamThreads), 0, s,
                     1u, scores, done, static_cast<const lmh::BeamPartial *>(part),
                     static_cast<const lmh::BeamCand *>(cand), o, static_cast<int32_t>(W),
                     static_cast<int32_t>(C), static_cast<int32_t>(bp.parts), eos, status);
}

lmh_status_t beam_reorder(void *const *states, int64_t num_states, const int32_t *parents, int64_t N,
                          int64_t W, int64_t entry_stride, int64_t beam_stride, int64_t run_bytes,
                          const int64_t *outer, const int64_t *outer_stride, int64_t num_outer,
                          int32_t *status, lmh_stream_t stream)
{
    if (!states || !parents || num_states < 1 || num_states > lmh::kReorderMaxStates || N < 1 ||
        N > 65535 || W < 1 || W > lmh::kBeamMaxWidth || run_bytes < 1 || num_outer < 0 || num_outer > 3 ||
        (num_outer > 0 && (!outer || !outer_stride)))
        return LMH_ERR_INVALID_ARG;
    if (!aligned(parents, 4))
        return LMH_ERR_MISALIGNED;
    // Elements of a state must not share memory: taken from the smallest
    // stride up, each dimension has to step over all that lies below it.
    int64_t ext[5], str[5];
    int nd = 0;
    ext[nd] = N, str[nd++] = entry_stride;
    ext[nd] = W, str[nd++] = beam_stride;
    for (int64_t i = 0; i < num_outer; ++i)
        ext[nd] = outer[i], str[nd++] = outer_stride[i];
    for (int i = 0; i < nd; ++i)
        if (ext[i] < 1 || ext[i] > kMaxDim)
            return LMH_ERR_INVALID_ARG;
    for (int i = 1; i < nd; ++i)
        for (int j = i; j > 0 && str[j] < str[j - 1]; --j) {
            const int64_t e = ext[j], t = str[j];
            ext[j] = ext[j - 1], str[j] = str[j - 1];
            ext[j - 1] = e, str[j - 1] = t;
        }
    constexpr int64_t kMaxSpan = int64_t{1} << 46;  // far beyond device memory; keeps the sums in range
    if (run_bytes > kMaxSpan)
        return LMH_ERR_INVALID_ARG;
    int64_t span = run_bytes;
    Geometry geometry;
    geometry.run = run_bytes;
    uint64_t align = static_cast<uint64_t>(run_bytes) | 16u;
    for (int i = 0; i < nd; ++i) {
        if (ext[i] == 1)
            continue;
        if (str[i] < span || str[i] > kMaxSpan / ext[i])
            return LMH_ERR_INVALID_ARG;
        geometry.extent[geometry.n] = ext[i];
        geometry.stride[geometry.n] = str[i];
        geometry.below[geometry.n++] = span;
        span += (ext[i] - 1) * str[i];
        align |= static_cast<uint64_t>(str[i]);
    }
    lmh::ReorderParams p{};
    for (int64_t i = 0; i < num_states; ++i) {
        if (!states[i])
            return LMH_ERR_INVALID_ARG;
        for (int64_t j = 0; j < i; ++j) {
            // what two states share would be moved twice, by blocks that do not wait for each other
            const uintptr_t a = reinterpret_cast<uintptr_t>(states[i]), b = reinterpret_cast<uintptr_t>(states[j]);
            const uintptr_t apart = a > b ? a - b : b - a;
            if (apart < static_cast<uintptr_t>(span) &&
                states_meet(geometry, static_cast<int64_t>(apart), geometry.n - 1))
                return LMH_ERR_INVALID_ARG;
        }
        p.state[i] = static_cast<uint8_t *>(states[i]);
        align |= reinterpret_cast<uintptr_t>(states[i]);
    }
    int64_t vec = static_cast<int64_t>(align & (~align + 1));  // largest power of two, at most 16
    const int64_t most = W <= 16 ? 16 : W <= 32 ? 8 : 4;       // registers of a column
    vec = vec < most ? vec : most;
    int64_t columns = run_bytes / vec;
    for (int64_t i = 0; i < 3; ++i) {
        p.outer[i] = i < num_outer ? static_cast<uint32_t>(outer[i]) : 1u;
        p.outer_stride[i] = i < num_outer ? outer_stride[i] : 0;
        if (columns > kMaxDim / static_cast<int64_t>(p.outer[i]))
            return LMH_ERR_INVALID_ARG;
        columns *= p.outer[i];
    }
    p.entry_stride = entry_stride;
    p.beam_stride = beam_stride;
    p.run_vecs = static_cast<uint32_t>(run_bytes / vec);
    p.columns = static_cast<uint32_t>(columns);
    p.W = static_cast<int32_t>(W);
    p.parents = parents;
    p.status = status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int ns = static_cast<int>(num_states);
    switch (vec) {
    case 16: return dispatch_reorder<uint4>(p, N, ns, s);
    case 8: return dispatch_reorder<uint2>(p, N, ns, s);
    case 4: return dispatch_reorder<uint32_t>(p, N, ns, s);
    case 2: return dispatch_reorder<uint16_t>(p, N, ns, s);
    default: return dispatch_reorder<uint8_t>(p, N, ns, s);
    }
}

}  // extern "C"
