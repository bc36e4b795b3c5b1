// A call of the 4-bit decode kernel, decode_q4.cuh (one file per head_dim).
#pragma once

#include "common.cuh"

namespace pkv {

struct Q4Decode {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;  // decode
  const int32_t* cu_q;          // chunks of at most 8 rows per KV head, or null
  const int32_t* cu_k;
  unsigned int* err;
  int max_blocks, batch, hq, hkv, block_size, num_blocks;
  int num_splits;
  int total_q, max_seqlen_q, causal;
  float scale, k_scale, v_scale;
  void* workspace;
  size_t workspace_bytes;
};

int decode_q4_d64(const Q4Decode& a, cudaStream_t stream);
int decode_q4_d128(const Q4Decode& a, cudaStream_t stream);

}  // namespace pkv
