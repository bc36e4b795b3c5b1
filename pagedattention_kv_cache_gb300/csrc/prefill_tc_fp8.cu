// The tcgen05 prefill (prefill_tc.cuh) over an FP8 E4M3 cache.
#include "prefill_tc.cuh"

namespace pkv {

int prefill_tc_fp8_launch(const PrefillArgs& a, cudaStream_t stream) { return launch_form<kE4m3>(a, stream); }

}  // namespace pkv
