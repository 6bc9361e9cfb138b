// host.cuh -- host-side helpers shared by the library's translation units:
// argument checks, the device's SM count, the tensor-map encoder and launches
// with programmatic stream serialisation.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "lmhead.h"

namespace lmh {
namespace host {

constexpr int64_t kMaxDim = 0x7fffffff;
constexpr int kMaxDevices = 64;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int num_sms()
{
    // per device, filled on first use; host threads may race to fill it, with the same value
    static std::atomic<int> cached[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return 148;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 148;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// cuTensorMapEncodeTiled, resolved once through the runtime (no -lcuda).
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 2-D BF16 tensor [outer, inner] (inner contiguous), 128-byte swizzled boxes
// of box_inner x box_outer elements; out-of-range elements read as zero.
inline bool make_map(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer,
              uint32_t box_inner, uint32_t box_outer)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {inner * 2};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output tensor map for the TMA-store epilogue: [outer rows][row stride ld]
// of FP32 or BF16, box {32, box_rows}, no swizzle.  False when the layout
// cannot be described (base not 16-byte aligned, row stride not a multiple
// of 16 bytes); the caller then uses the direct-store epilogue.
inline bool make_out_map(CUtensorMap *map, void *base, bool bf16, uint64_t inner, uint64_t outer,
                  uint64_t ld, uint32_t box_rows)
{
    const uint64_t esize = bf16 ? 2 : 4;
    if (!aligned(base, 16) || (ld * esize) % 16 != 0)
        return false;
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {ld * esize};
    const cuuint32_t box[2] = {32, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base,
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline lmh_status_t last_cuda_error()
{
    return cudaGetLastError() == cudaSuccess ? LMH_OK : LMH_ERR_CUDA;
}

// Programmatic dependent launch is on unless the library is built with
// -DLMH_NO_PDL (a build-time switch for measurements; nothing in the
// environment changes the kernels a call launches).
constexpr bool pdl_enabled()
{
#ifdef LMH_NO_PDL
    return false;
#else
    return true;
#endif
}

// Launch with programmatic stream serialisation allowed (the kernel waits in
// pdl_wait before touching memory the previous kernel may still write) and,
// for cluster_x > 1, thread-block clusters of cluster_x CTAs.
template <typename... KArgs, typename... Args>
lmh_status_t launch_ex(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, unsigned cluster_x, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (pdl_enabled()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    if (cluster_x > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster_x;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess)
        return LMH_ERR_CUDA;
    return last_cuda_error();
}

inline bool bad_dtype(int32_t t) { return t != LMH_F32 && t != LMH_BF16; }

inline bool dims_ok(int64_t a, int64_t b, int64_t c)
{
    return a >= 1 && b >= 1 && c >= 1 && a <= kMaxDim && b <= kMaxDim && c <= kMaxDim;
}

}  // namespace host
}  // namespace lmh
