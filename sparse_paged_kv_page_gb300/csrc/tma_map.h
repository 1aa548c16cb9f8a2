// Host side: tensor maps of the paged pools for the TMA engine.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "sparse_attn.h"

namespace sa {

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);
// Looked up by the first call; calls of other threads wait for it.
inline EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                           cudaSuccess &&
                       q == cudaDriverEntryPointSuccess;
    return found ? reinterpret_cast<EncodeFn>(p) : nullptr;
  }();
  return fn;
}

// Tensor map over every pool row: [rows = num_blocks * H * page_size, D], box box_rows x 64, 128-byte swizzle.
inline bool make_pool_map(CUtensorMap* m, const void* base, const sa_cache* c, int box_rows) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t rows = cuuint64_t(c->num_blocks) * c->num_kv_heads * c->page_size;
  if (rows >= (cuuint64_t(1) << 31)) return false;
  const cuuint64_t dims[2] = {cuuint64_t(c->head_dim), rows};
  const cuuint64_t strides[1] = {cuuint64_t(c->head_dim) * 2};
  const cuuint32_t box[2] = {64, cuuint32_t(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over every pool row as groups of 8 rows of 64-column halves: (64, 8, D / 64, rows / 8). One box is a
// whole page of a head, `groups` of 8 rows: in shared memory [group][half][8 rows of 128 bytes], 128-byte swizzle.
// One box for both halves matters: a copy costs the TMA engine about 100 cycles below 4 KB, whatever its size.
inline bool make_group_map(CUtensorMap* m, const void* base, const sa_cache* c, int groups) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t rows = cuuint64_t(c->num_blocks) * c->num_kv_heads * c->page_size;
  if (rows >= (cuuint64_t(1) << 31)) return false;
  const cuuint64_t row = cuuint64_t(c->head_dim) * 2;
  const cuuint64_t dims[4] = {64, 8, cuuint64_t(c->head_dim) / 64, rows / 8};
  const cuuint64_t strides[3] = {row, 128, 8 * row};
  const cuuint32_t box[4] = {64, 8, cuuint32_t(c->head_dim) / 64, cuuint32_t(groups)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over every pool row, both 64-column halves in one box of 16 rows: (64, rows, D / 64), in shared memory
// [half][16 rows of 128 bytes], 128-byte swizzle.
inline bool make_row_map(CUtensorMap* m, const void* base, const sa_cache* c) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t rows = cuuint64_t(c->num_blocks) * c->num_kv_heads * c->page_size;
  if (rows >= (cuuint64_t(1) << 31)) return false;
  const cuuint64_t dims[3] = {64, rows, cuuint64_t(c->head_dim) / 64};
  const cuuint64_t strides[2] = {cuuint64_t(c->head_dim) * 2, 128};
  const cuuint32_t box[3] = {64, 16, cuuint32_t(c->head_dim) / 64};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of query rows [tokens, heads, D], box `box_tokens` x `box_heads` x 64 columns, 128-byte swizzle.
inline bool make_query_map(CUtensorMap* m, const void* base, int D, int heads, int tokens, int box_heads,
                           int box_tokens) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(heads), cuuint64_t(tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(D) * 2 * heads};
  const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sa
