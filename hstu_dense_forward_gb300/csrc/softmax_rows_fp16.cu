// Softmax attention of few fp16 query rows.
#include "softmax_rows.cuh"

namespace hstu {

cudaError_t launch_softmax_rows_fp16(const SoftmaxParams& p, bool e4m3, const CUtensorMap& tc,
                                    int rows, long long tiles, long long blocks, int cluster,
                                    cudaStream_t stream) {
  return e4m3 ? rows::launch_rows<false, true>(p, tc, rows, tiles, blocks, cluster, stream)
              : rows::launch_rows<false, false>(p, tc, rows, tiles, blocks, cluster, stream);
}

}  // namespace hstu
