// The tcgen05 prefill (prefill_tc.cuh) with document, window or prefix masks.
#include "prefill_tc.cuh"

namespace pkv {

int prefill_tc_masked_launch(const PrefillArgs& a, cudaStream_t stream) { return launch_form<kMasked>(a, stream); }

}  // namespace pkv
