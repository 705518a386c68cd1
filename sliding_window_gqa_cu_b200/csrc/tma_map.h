// Host helpers shared by the entry points: TMA descriptor encoding for the
// packed [T, H, D] bf16 tensors and the 16-byte alignment check.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

namespace thd {

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult qr{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &qr) ==
                cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// 3-D map over a [T, H, D] bf16 tensor: dims (D, H, T), box (64, 1, rows),
// 128-byte swizzle; out-of-range rows read as zero.
inline bool make_map(CUtensorMap* map, const void* base, int64_t T, int H, int D, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                          static_cast<cuuint64_t>(T)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H) * D * 2};
    cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 5-D map over a paged bf16 cache [blocks, block, H, D] with D dense and the
// given token stride: dims (64 columns, 8 tokens, D / 64 column chunks, block / 8,
// places), where place n begins n * place_stride elements into the cache (its
// blocks and heads; a place outside reads as zero).  Box (64, 8, box_chunks,
// box_rows / 8, 1), 128-byte swizzle.
inline bool make_paged_map(CUtensorMap* map, const void* base, int block, int D, int64_t token_stride,
                           int64_t place_stride, int64_t places, int box_rows, int box_chunks) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(D) / 64, static_cast<cuuint64_t>(block) / 8,
                          static_cast<cuuint64_t>(places)};
    cuuint64_t strides[4] = {static_cast<cuuint64_t>(token_stride) * 2, 128, static_cast<cuuint64_t>(token_stride) * 16,
                             static_cast<cuuint64_t>(place_stride) * 2};
    cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(box_chunks), static_cast<cuuint32_t>(box_rows / 8), 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace thd
