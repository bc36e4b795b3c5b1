// The tcgen05 prefill (prefill_tc.cuh) with a distance bias.
#include "prefill_tc.cuh"

namespace pkv {

int prefill_tc_biased_launch(const PrefillArgs& a, cudaStream_t stream) { return launch_form<kBiased>(a, stream); }

}  // namespace pkv
