// The 4-bit decode kernel (decode_q4.cuh) at head_dim 64.
#include "decode_q4.cuh"

namespace pkv {

int decode_q4_d64(const Q4Decode& a, cudaStream_t stream) { return run_q4<64>(a, stream); }

}  // namespace pkv
