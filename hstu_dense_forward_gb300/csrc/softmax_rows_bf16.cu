// Softmax attention of few bf16 query rows.
#include "softmax_rows.cuh"

namespace hstu {

cudaError_t launch_softmax_rows_bf16(const SoftmaxParams& p, int fmt, const CUtensorMap& tc,
                                    int rows, long long tiles, long long blocks, int cluster,
                                    cudaStream_t stream) {
  return fmt == kE4m3   ? rows::launch_rows<true, kE4m3>(p, tc, rows, tiles, blocks, cluster, stream)
         : fmt == kE2m1 ? rows::launch_rows<true, kE2m1>(p, tc, rows, tiles, blocks, cluster, stream)
                        : rows::launch_rows<true, kSame>(p, tc, rows, tiles, blocks, cluster, stream);
}

}  // namespace hstu
