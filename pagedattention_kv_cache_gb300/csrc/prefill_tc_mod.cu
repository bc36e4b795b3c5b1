// The tcgen05 prefill (prefill_tc.cuh) with score modifiers.
#include "prefill_tc.cuh"

namespace pkv {

int prefill_tc_mod_launch(const PrefillArgs& a, cudaStream_t stream) {
  return a.head_dim == 64 ? launch_d<64, true, false>(a, stream) : launch_d<128, true, false>(a, stream);
}

}  // namespace pkv
