// Tensor-core softmax attention: fp16 queries over an E4M3 cache.
#include "softmax_tc.cuh"

namespace hstu {

cudaError_t launch_softmax_tc_fp16_e4m3(const SoftmaxParams& p, const CUtensorMap& tq,
                                 const CUtensorMap& tc, int qtiles, int ctas, long long tiles,
                                 long long blocks, cudaStream_t stream) {
  return sm::launch_tc<false, kE4m3>(p, tq, tc, qtiles, ctas, tiles, blocks, stream);
}

}  // namespace hstu
