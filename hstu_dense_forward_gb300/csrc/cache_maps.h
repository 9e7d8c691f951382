// Tensor maps of the paged KV cache and of the queries over it.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "kv_cache.cuh"
#include "tensor_map.h"

namespace hstu {

// Head dim of the kernel that runs D: rows shorter than it are filled with zeros by TMA.
inline int kernel_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

inline CUtensorMapDataType elem_type(int dtype) {
  return dtype == HSTU_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// The cache [num_pages, 2, page_size, Nk, D] in boxes of `inner` elements and up to `rows`
// rows of one page, with rows of `swizzle` bytes (0: none).
inline bool cache_map(CUtensorMap* m, const SoftmaxParams& p, int dtype, bool e4m3, int inner, int rows,
               int swizzle) {
  const EncodeTiledFn encode = encode_fn();
  const cuuint64_t D = (cuuint64_t)p.c.D, Nk = (cuuint64_t)p.c.Nk, eb = e4m3 ? 1 : 2;
  const cuuint64_t ps = 1ull << p.c.page_shift;
  const cuuint64_t dims[4] = {D, Nk, ps, 2 * (cuuint64_t)p.c.num_pages};
  const cuuint64_t strides[3] = {D * eb, Nk * D * eb, ps * Nk * D * eb};
  const cuuint32_t box[4] = {(cuuint32_t)inner, 1,
                             (cuuint32_t)(ps < (cuuint64_t)rows ? ps : rows), 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return encode &&
         encode(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : elem_type(dtype), 4, p.c.cache, dims,
                strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                swizzle == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                : swizzle == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The E2M1 cache [num_pages, 2, Nk, page_size, D / 2] in boxes of `inner` bytes and up to `rows`
// rows of one head and page.
inline bool code_map(CUtensorMap* m, const SoftmaxParams& p, int inner, int rows, int swizzle) {
  const EncodeTiledFn encode = encode_fn();
  const cuuint64_t row = (cuuint64_t)p.c.D / 2, ps = 1ull << p.c.page_shift;
  const cuuint64_t dims[4] = {row, ps, (cuuint64_t)p.c.Nk, 2 * (cuuint64_t)p.c.num_pages};
  const cuuint64_t strides[3] = {row, row * ps, row * ps * p.c.Nk};
  const cuuint32_t box[4] = {(cuuint32_t)inner, (cuuint32_t)(ps < (cuuint64_t)rows ? ps : rows), 1,
                             1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return encode &&
         encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.c.cache, dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                swizzle == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                : swizzle == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries [T, Nq, D]: the G heads of one kv head of 128 / G tokens make one tile of packed rows.
inline bool query_map(CUtensorMap* m, const SoftmaxParams& p, int dtype) {
  const EncodeTiledFn encode = encode_fn();
  const cuuint64_t dims[3] = {(cuuint64_t)p.c.D, (cuuint64_t)p.Nq, (cuuint64_t)p.c.T};
  const cuuint64_t strides[2] = {(cuuint64_t)p.c.D * 2, (cuuint64_t)p.q_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(128 / p.G)};
  const cuuint32_t one[3] = {1, 1, 1};
  return encode &&
         encode(m, elem_type(dtype), 3, const_cast<void*>(p.q), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace hstu
