// Tensor maps and the choice of translation unit for the attention weights of cached keys.
#include <cuda.h>
#include <cuda_runtime.h>

#include "cache_maps.h"
#include "evict_kernels.h"

namespace hstu {

#define HSTU_WEIGHTS_UNITS(n)                                                                 \
  cudaError_t launch_weights_rows_##n(const WeightsParams& w, int fmt, const CUtensorMap& tc, \
                                      int rows, cudaStream_t s);                              \
  cudaError_t launch_weights_tc_##n(const WeightsParams& w, int fmt, const CUtensorMap& tq,   \
                                    const CUtensorMap& tc, int slots, int cluster,            \
                                    cudaStream_t s)
HSTU_WEIGHTS_UNITS(bf16);
HSTU_WEIGHTS_UNITS(fp16);
#undef HSTU_WEIGHTS_UNITS

int weights_rows_ctas(int D, int fmt, int rows) {
  const int dim = kernel_dim(D), row = fmt == kE2m1 ? dim / 2 : fmt == kE4m3 ? dim : 2 * dim;
  if (row == 512 || (dim == 256 && rows == 16)) return 1;
  return row > 128 || dim == 256 || rows == 16 ? 2 : 3;
}

int weights_tc_keys(int D) { return kernel_dim(D) == 256 ? 128 : 256; }

cudaError_t launch_weights_rows(const WeightsParams& w, int dtype, int fmt, int rows,
                                cudaStream_t stream) {
  CUtensorMap tc;
  const bool e4m3 = fmt == kE4m3;
  const int row_bytes =
      fmt == kE2m1 ? kernel_dim(w.a.c.D) / 2 : kernel_dim(w.a.c.D) * (e4m3 ? 1 : 2);
  const int swz = row_bytes < 128 ? row_bytes : 128;
  if (!(fmt == kE2m1 ? code_map(&tc, w.a, swz, 128, swz)
                     : cache_map(&tc, w.a, dtype, e4m3, swz / (e4m3 ? 1 : 2), 128, swz)))
    return cudaErrorInvalidValue;
  return dtype == HSTU_BF16 ? launch_weights_rows_bf16(w, fmt, tc, rows, stream)
                            : launch_weights_rows_fp16(w, fmt, tc, rows, stream);
}

cudaError_t launch_weights_tc(const WeightsParams& w, int dtype, int fmt, int slots, int cluster,
                              cudaStream_t stream) {
  CUtensorMap tq, tc = {};
  if (!query_map(&tq, w.a, dtype)) return cudaErrorInvalidValue;
  // (the keys of other caches are converted, from plain loads)
  if (fmt == kSame && !cache_map(&tc, w.a, dtype, false, 64, 128, 128))
    return cudaErrorInvalidValue;
  return dtype == HSTU_BF16 ? launch_weights_tc_bf16(w, fmt, tq, tc, slots, cluster, stream)
                            : launch_weights_tc_fp16(w, fmt, tq, tc, slots, cluster, stream);
}

}  // namespace hstu
