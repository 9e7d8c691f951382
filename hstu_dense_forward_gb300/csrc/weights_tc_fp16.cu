// Attention weights of the cached keys from fp16 queries, on the tensor cores.
#include "weights_tc.cuh"

namespace hstu {

cudaError_t launch_weights_tc_fp16(const WeightsParams& w, int fmt, const CUtensorMap& tq,
                                  const CUtensorMap& tc, int slots, int cluster, cudaStream_t s) {
  return fmt == kE4m3   ? wt::launch_dim<false, kE4m3>(w, tq, tc, slots, cluster, s)
         : fmt == kE2m1 ? wt::launch_dim<false, kE2m1>(w, tq, tc, slots, cluster, s)
                        : wt::launch_dim<false, kSame>(w, tq, tc, slots, cluster, s);
}

}  // namespace hstu
