// Attention weights of the cached keys from few fp16 query rows.
#include "weights_rows.cuh"

namespace hstu {

cudaError_t launch_weights_rows_fp16(const WeightsParams& w, int fmt, const CUtensorMap& tc, int rows,
                                   cudaStream_t s) {
  return fmt == kE4m3   ? rows::launch_weights_fmt<false, kE4m3>(w, tc, rows, s)
         : fmt == kE2m1 ? rows::launch_weights_fmt<false, kE2m1>(w, tc, rows, s)
                        : rows::launch_weights_fmt<false, kSame>(w, tc, rows, s);
}

}  // namespace hstu
