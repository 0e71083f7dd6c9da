// Host side of the TMA tiled copies: the driver's tensor-map encoder, looked up
// once through the runtime (no link against libcuda), and a 2-D map builder.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

namespace kda {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// 2-D map over a [rows][row_elems] row-major tensor, box = box_cols x box_rows
inline cudaError_t make_map(CUtensorMap* m, CUtensorMapDataType dt, size_t esize, const void* ptr,
                            uint64_t row_elems, uint64_t rows, uint32_t box_cols, uint32_t box_rows,
                            CUtensorMapSwizzle sw) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {row_elems, rows < 1 ? 1 : rows};
    cuuint64_t strides[1] = {row_elems * esize};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t es[2] = {1, 1};
    CUresult r = enc(m, dt, 2, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// 3-D map over a [rows][heads][d] bf16 tensor whose tokens are row_stride elements
// apart, box = box_cols (64 or 32) channels x box_heads x box_rows, swizzled over its rows of
// 128 or 64 bytes
inline cudaError_t make_map_heads(CUtensorMap* m, const void* ptr, uint64_t d, uint64_t heads, uint64_t rows,
                                  uint64_t row_stride, uint32_t box_heads, uint32_t box_rows, uint32_t box_cols = 64) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[3] = {d, heads, rows < 1 ? 1 : rows};
    cuuint64_t strides[2] = {d * 2, row_stride * 2};
    cuuint32_t box[3] = {box_cols, box_heads, box_rows};
    cuuint32_t es[3] = {1, 1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace kda
