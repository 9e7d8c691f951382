// Tensor maps and the choice of translation unit for the 16-bit softmax attention kernels.
#include <cuda.h>
#include <cuda_runtime.h>

#include "cache_maps.h"
#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"

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

int softmax_rows_ctas(int D, int fmt, int rows) {
  const bool wide = kernel_dim(D) == 256, more = fmt != kSame && rows == 8;
  return wide ? (more ? 2 : 1) : (more ? 3 : 2);
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
  if (!encode_fn()) return cudaErrorNotSupported;
  CUtensorMap tq = {}, tc;
  if (kernel_dim(p.c.D) == 128 && (qtiles == 2 || ctas == 2)) {  // queries by TMA:
    // the G heads of one kv head of 128 / G tokens make one tile of packed rows
    if (!query_map(&tq, p, dtype)) return cudaErrorInvalidValue;
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
