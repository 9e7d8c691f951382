// Tensor maps and the choice of translation unit for the 16-bit softmax attention kernels.
#include <cuda.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"
#include "tensor_map.h"

namespace hstu {

#define HSTU_TC_UNIT(n)                                                                       \
  cudaError_t launch_softmax_tc_##n(const SoftmaxParams& p, const CUtensorMap& tq,            \
                                    const CUtensorMap& tc, int qtiles, int ctas,              \
                                    long long tiles, long long blocks, cudaStream_t stream)
HSTU_TC_UNIT(bf16);
HSTU_TC_UNIT(fp16);
HSTU_TC_UNIT(bf16_e4m3);
HSTU_TC_UNIT(fp16_e4m3);
HSTU_TC_UNIT(bf16_e2m1);
HSTU_TC_UNIT(fp16_e2m1);
#undef HSTU_TC_UNIT
#define HSTU_ROWS_UNIT(n)                                                                     \
  cudaError_t launch_softmax_rows_##n(const SoftmaxParams& p, int fmt,                        \
                                      const CUtensorMap& tc, int rows, long long tiles,       \
                                      long long blocks, int cluster, cudaStream_t stream)
HSTU_ROWS_UNIT(bf16);
HSTU_ROWS_UNIT(fp16);
#undef HSTU_ROWS_UNIT

namespace {

// Head dim of the kernel that runs D: rows shorter than it are filled with zeros by TMA.
int kernel_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

CUtensorMapDataType elem_type(int dtype) {
  return dtype == HSTU_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// The cache [num_pages, 2, page_size, Nk, D] in boxes of `inner` elements and up to `rows`
// rows of one page, with rows of `swizzle` bytes (0: none).
bool cache_map(CUtensorMap* m, const SoftmaxParams& p, int dtype, bool e4m3, int inner, int rows,
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
bool code_map(CUtensorMap* m, const SoftmaxParams& p, int inner, int rows, int swizzle) {
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

}  // namespace

int softmax_rows_ctas(int D, int fmt, int rows) {
  const bool more = fmt != kSame && rows == 8;
  return kernel_dim(D) == 256 ? (more ? 2 : 1) : (more ? 3 : 2);
}

cudaError_t launch_softmax_rows(const SoftmaxParams& p, int dtype, int fmt, int rows,
                                long long tiles, long long blocks, int cluster,
                                cudaStream_t stream) {
  CUtensorMap tc;
  const bool e4m3 = fmt == kE4m3;
  const int row_bytes =
      fmt == kE2m1 ? kernel_dim(p.c.D) / 2 : kernel_dim(p.c.D) * (e4m3 ? 1 : 2);
  const int swz = row_bytes < 128 ? row_bytes : 128;
  if (!(fmt == kE2m1 ? code_map(&tc, p, swz, 64, swz)
                     : cache_map(&tc, p, dtype, e4m3, swz / (e4m3 ? 1 : 2), 64, swz)))
    return cudaErrorInvalidValue;
  return dtype == HSTU_BF16
             ? launch_softmax_rows_bf16(p, fmt, tc, rows, tiles, blocks, cluster, stream)
             : launch_softmax_rows_fp16(p, fmt, tc, rows, tiles, blocks, cluster, stream);
}

cudaError_t launch_softmax_tc(const SoftmaxParams& p, int dtype, int fmt, int qtiles, int ctas,
                              long long tiles, long long blocks, cudaStream_t stream) {
  const EncodeTiledFn encode = encode_fn();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap tq = {}, tc;
  if (kernel_dim(p.c.D) == 128 && (qtiles == 2 || ctas == 2)) {  // queries by TMA:
    // the G heads of one kv head of 128 / G tokens make one tile of packed rows
    const cuuint64_t dims[3] = {(cuuint64_t)p.c.D, (cuuint64_t)p.Nq, (cuuint64_t)p.c.T};
    const cuuint64_t strides[2] = {(cuuint64_t)p.c.D * 2, (cuuint64_t)p.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(128 / p.G)};
    const cuuint32_t one[3] = {1, 1, 1};
    if (encode(&tq, elem_type(dtype), 3, const_cast<void*>(p.q), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  // rows of codes are staged whole and unswizzled
  const bool e4m3 = fmt == kE4m3;
  const int kt = kernel_dim(p.c.D) == 256 ? 64 : 128;
  if (!(fmt == kE2m1 ? code_map(&tc, p, kernel_dim(p.c.D) / 2, kt, 0)
                     : cache_map(&tc, p, dtype, e4m3, e4m3 ? kernel_dim(p.c.D) : 64, kt,
                                 e4m3 ? 0 : 128)))
    return cudaErrorInvalidValue;
  auto* launch = dtype == HSTU_BF16
                     ? (fmt == kE4m3   ? launch_softmax_tc_bf16_e4m3
                        : fmt == kE2m1 ? launch_softmax_tc_bf16_e2m1
                                       : launch_softmax_tc_bf16)
                     : (fmt == kE4m3   ? launch_softmax_tc_fp16_e4m3
                        : fmt == kE2m1 ? launch_softmax_tc_fp16_e2m1
                                       : launch_softmax_tc_fp16);
  return launch(p, tq, tc, qtiles, ctas, tiles, blocks, stream);
}

}  // namespace hstu
