// Softmax attention of few fp16 query rows.
#include "softmax_rows.cuh"

namespace hstu {

cudaError_t launch_softmax_rows_fp16(const SoftmaxParams& p, int fmt, const CUtensorMap& tc,
                                    int rows, long long tiles, long long blocks, int cluster,
                                    cudaStream_t stream) {
  return fmt == kE4m3   ? rows::launch_rows<false, kE4m3>(p, tc, rows, tiles, blocks, cluster, stream)
         : fmt == kE2m1 ? rows::launch_rows<false, kE2m1>(p, tc, rows, tiles, blocks, cluster, stream)
                        : rows::launch_rows<false, kSame>(p, tc, rows, tiles, blocks, cluster, stream);
}

}  // namespace hstu
