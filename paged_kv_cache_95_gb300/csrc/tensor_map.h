// tensor_map.h -- the driver's tensor-map encoder, looked up once, and the maps of the K/V pools.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "launch.h"

namespace pkv {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// An FP8 pool [num_blocks][n_kv][16][128] of one-byte codes viewed as 4-D; one box
// = a whole 2 KB (block, head) tile (128 codes = 128 bytes x 16 slots), 128-byte swizzle.
inline bool encode_pool_map_fp8(CUtensorMap *map, const void *base, int32_t num_blocks, int32_t n_kv) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(kBlockSize),
                                static_cast<cuuint64_t>(n_kv), static_cast<cuuint64_t>(num_blocks)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(kHeadDim) * kBlockSize,
                                   static_cast<cuuint64_t>(kHeadDim) * kBlockSize * n_kv};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(kHeadDim), static_cast<cuuint32_t>(kBlockSize), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same pool viewed as 5-D so that ONE box is a whole 4 KB (block, head) tile
// in the order the tensor core wants it: dims inner->outer are 64 dims (128 B),
// 8 slots (stride 256 B), the two 64-dim halves (stride 128 B), the two 8-slot
// groups (stride 2 KB) and the (block, head) tile index block * n_kv + head
// (stride 4 KB).  The box (64, 8, 2, 2, 1) lands in shared memory as
// [slot group][dim half][8 slots][128 B], i.e. four 1 KB swizzle atoms.
inline bool encode_pool_tile_map(CUtensorMap *map, const void *base, int32_t num_blocks, int32_t n_kv) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const uint64_t tiles = static_cast<uint64_t>(num_blocks) * static_cast<uint64_t>(n_kv);
    if (tiles > static_cast<uint64_t>(INT32_MAX)) return false;  // tile index is a 32-bit coordinate
    const cuuint64_t dims[5] = {64, 8, 2, 2, static_cast<cuuint64_t>(tiles)};
    const cuuint64_t strides[4] = {256, 128, 2048, 4096};
    const cuuint32_t box[5] = {64, 8, 2, 2, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows [rows][n_q][128] of bf16; a box (64 values, `group` heads, 128 / group rows) lands as 128 lines of 128 bytes,
// 128-byte swizzle: one value half of the heads of a KV head, row after row.
inline bool encode_query_group_map(CUtensorMap *map, const void *base, int32_t rows, int32_t n_q, int32_t group) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(n_q), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {2ull * kHeadDim, 2ull * kHeadDim * n_q};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(128 / group)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pkv
