// Tensor maps on the host, through the driver entry point (no libcuda link).  (gemm.cu keeps
// its own copies: recorded traffic measurements are matched to that file by its hash.)
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace mxmoe {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// Row-major uint8 matrix [rows, row_bytes] read in boxes of 128 bytes x box_rows,
// 128-byte swizzle.
inline cudaError_t make_tmap(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows,
                      uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Packed E2M1 matrix [rows, K elements] (K/2 bytes a row), read in boxes of 128
// elements x 128 rows that land one element per byte: each 16 elements' 8 packed
// bytes followed by 8 unused bytes (CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B), the
// operand layout of kind::mxf8f6f4 for E2M1; 128-byte swizzle, 16 KiB a box.
inline cudaError_t make_tmap_e2m1_wide(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {K, rows};
  const cuuint64_t strides[1] = {K / 2};
  const cuuint32_t box[2] = {128, kBM};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<void*>(base),
                         dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// 128x4 scale blocks of `row_blocks` 128-row groups of `per_row` 512-byte blocks each, as
// 256-byte rows in three dimensions, read `blocks` along K by `rows` groups at a time;
// blocks past the end read as zeros.
inline cudaError_t make_tmap_scales(CUtensorMap* m, const void* base, uint64_t per_row,
                                    uint64_t row_blocks, uint32_t blocks, uint32_t rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {256, 2 * per_row, row_blocks};
  const cuuint64_t strides[2] = {256, 512 * per_row};
  const cuuint32_t box[3] = {256, 2 * blocks, rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// bf16 rows of D elements (64 or 128) read in boxes of 64 elements x box_rows, 128-byte swizzle;
// rows past the end read as zeros.
inline cudaError_t make_tmap_bf16(CUtensorMap* m, const void* base, uint64_t D, uint64_t rows,
                                  uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {D, rows};
  const cuuint64_t strides[1] = {2 * D};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// bf16 heads [tokens, heads, D] with `ld` elements from token to token, read in boxes of 64
// elements x box_heads x box_tokens that land as rows of 128 bytes, 128-byte swizzle.
inline cudaError_t make_tmap_heads(CUtensorMap* m, const void* base, uint64_t D, uint64_t heads,
                                   uint64_t tokens, uint64_t ld, uint32_t box_heads,
                                   uint32_t box_tokens) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {D, heads, tokens};
  const cuuint64_t strides[2] = {2 * D, 2 * ld};
  const cuuint32_t box[3] = {64, box_heads, box_tokens};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace mxmoe
