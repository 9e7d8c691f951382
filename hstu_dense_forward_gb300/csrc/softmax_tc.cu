// Tensor maps and the choice of translation unit for the tensor-core softmax attention.
#include <cuda.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"
#include "tensor_map.h"

namespace hstu {

#define HSTU_TC_UNIT(n)                                                                       \
  cudaError_t launch_softmax_tc_##n(const SoftmaxParams& p, const CUtensorMap& tq,            \
                                    const CUtensorMap& tc, int qtiles, long long tiles,       \
                                    long long blocks, cudaStream_t stream)
HSTU_TC_UNIT(bf16);
HSTU_TC_UNIT(fp16);
HSTU_TC_UNIT(bf16_e4m3);
HSTU_TC_UNIT(fp16_e4m3);
#undef HSTU_TC_UNIT

namespace {

// Head dim of the kernel that runs D: rows shorter than it are filled with zeros by TMA.
int kernel_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

}  // namespace

int softmax_tc_key_tile(int D) { return kernel_dim(D) == 256 ? 64 : 128; }

cudaError_t launch_softmax_tc(const SoftmaxParams& p, int dtype, bool e4m3, int qtiles,
                              long long tiles, long long blocks, cudaStream_t stream) {
  const EncodeTiledFn encode = encode_fn();
  if (!encode) return cudaErrorNotSupported;
  const CUtensorMapDataType ty = dtype == HSTU_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t D = (cuuint64_t)p.c.D, Nk = (cuuint64_t)p.c.Nk;
  const cuuint64_t ps = 1ull << p.c.page_shift;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  CUtensorMap tq, tc;
  // queries: the G heads of one kv head of 128 / G tokens make one tile of packed rows
  {
    const cuuint64_t dims[3] = {D, (cuuint64_t)p.Nq, (cuuint64_t)p.c.T};
    const cuuint64_t strides[2] = {D * 2, (cuuint64_t)p.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(128 / p.G)};
    if (encode(&tq, ty, 3, const_cast<void*>(p.q), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  // the cache [num_pages, 2, page_size, Nk, D]; E4M3 rows are staged whole and unswizzled
  {
    const cuuint64_t eb = e4m3 ? 1 : 2;
    const cuuint64_t kt = (cuuint64_t)softmax_tc_key_tile(p.c.D);
    const cuuint64_t dims[4] = {D, Nk, ps, 2 * (cuuint64_t)p.c.num_pages};
    const cuuint64_t strides[3] = {D * eb, Nk * D * eb, ps * Nk * D * eb};
    const cuuint32_t box[4] = {e4m3 ? (cuuint32_t)kernel_dim(p.c.D) : 64u, 1,
                               (cuuint32_t)(ps < kt ? ps : kt), 1};
    if (encode(&tc, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : ty, 4, p.c.cache, dims, strides, box,
               one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (dtype == HSTU_BF16)
    return e4m3 ? launch_softmax_tc_bf16_e4m3(p, tq, tc, qtiles, tiles, blocks, stream)
                : launch_softmax_tc_bf16(p, tq, tc, qtiles, tiles, blocks, stream);
  return e4m3 ? launch_softmax_tc_fp16_e4m3(p, tq, tc, qtiles, tiles, blocks, stream)
              : launch_softmax_tc_fp16(p, tq, tc, qtiles, tiles, blocks, stream);
}

}  // namespace hstu
