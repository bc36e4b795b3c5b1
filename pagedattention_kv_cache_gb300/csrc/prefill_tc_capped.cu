// The tcgen05 prefill (prefill_tc.cuh) with capped scores.
#include "prefill_tc.cuh"

namespace pkv {

int prefill_tc_capped_launch(const PrefillArgs& a, cudaStream_t stream) { return launch_form<kCapped>(a, stream); }

}  // namespace pkv
