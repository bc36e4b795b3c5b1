// The tcgen05 prefill (prefill_tc.cuh) over a 4-bit cache.
#include "prefill_tc.cuh"

namespace pkv {

int prefill_tc_q4_launch(const PrefillArgs& a, cudaStream_t stream) { return launch_form<kInt4>(a, stream); }

}  // namespace pkv
