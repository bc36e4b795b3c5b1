// The tcgen05 prefill (prefill_tc.cuh) with capped scores and a distance bias.
#include "prefill_tc.cuh"

namespace pkv {

int prefill_tc_capped_biased_launch(const PrefillArgs& a, cudaStream_t stream) { return launch_form<kCappedBiased>(a, stream); }

}  // namespace pkv
