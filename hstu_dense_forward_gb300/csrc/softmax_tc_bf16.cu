// Tensor-core softmax attention: bf16 queries over a cache of the same type.
#include "softmax_tc.cuh"

namespace hstu {

cudaError_t launch_softmax_tc_bf16(const SoftmaxParams& p, const CUtensorMap& tq,
                                 const CUtensorMap& tc, int qtiles, int ctas, long long tiles,
                                 long long blocks, cudaStream_t stream) {
  return sm::launch_tc<true, kSame>(p, tq, tc, qtiles, ctas, tiles, blocks, stream);
}

}  // namespace hstu
