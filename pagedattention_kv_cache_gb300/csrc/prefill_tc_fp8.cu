// The tcgen05 prefill (prefill_tc.cuh) over an FP8 E4M3 cache.
#include "prefill_tc.cuh"

namespace pkv {

int prefill_tc_fp8_launch(const PrefillArgs& a, cudaStream_t stream) {
  return a.head_dim == 64 ? launch_d<64, false, true>(a, stream) : launch_d<128, false, true>(a, stream);
}

}  // namespace pkv
