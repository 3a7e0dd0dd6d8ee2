// tensor_maps.h -- host side of the chunk attention's TMA descriptors and
// kernel attributes.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "cache_common.cuh"

namespace k3da_chunk {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static std::mutex mutex;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::lock_guard<std::mutex> lock(mutex);
    if (fn == nullptr) {
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    return fn;
}

// Lets `kernel` have `bytes` of dynamic shared memory, once per device.
template <int SLOT>
inline bool allow_smem(const void *kernel, int bytes) {
    static std::mutex mutex;
    static uint64_t done[4] = {0, 0, 0, 0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return false;
    std::lock_guard<std::mutex> lock(mutex);
    if (done[dev / 64] >> (dev % 64) & 1) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done[dev / 64] |= 1ull << (dev % 64);
    return true;
}

// A pool as rows of 64 dims, in boxes of a page's 64 slots: bf16 with the
// 128-byte swizzle, codes as they lie or with the 64-byte swizzle.
inline bool pool_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *map, const void *pool, long long num_pages,
                     int hkv, bool quant, bool swizzled) {
    using namespace k3da_cache;
    const cuuint64_t dims[2] = {kD, static_cast<cuuint64_t>(num_pages) * 2 * hkv * kP};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD) * (quant ? 1 : 2)};
    const cuuint32_t box[2] = {kD, kP}, estrides[2] = {1, 1};
    return encode(map, quant ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  const_cast<void *>(pool), dims, strides, box, estrides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : quant ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace k3da_chunk
