// Arguments shared by the prefill kernels and their C entry points.
#pragma once

#include "common.cuh"
#include "score_mod.cuh"

namespace pkv {

struct PrefillArgs {
  void* out;
  const void* q;
  const void* k;
  const void* v;
  const void* k_cache;
  const void* v_cache;
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* block_tables;  // null: keys from the packed k, v
  unsigned int* err;
  int total_q;  // rows of q / out
  int total_k;  // rows of the packed k / v (0 when block_tables is used)
  int max_seqlen_q;
  int max_blocks;
  int batch;
  int hq;
  int hkv;
  int block_size;
  int num_blocks;
  float scale;
  int causal;
  int group;     // hq / hkv
  int head_dim;  // 64 or 128 (the mma.sync kernel: 128 only)
  void* workspace;         // split of long items (tcgen05 path), or null
  size_t workspace_bytes;
  float k_scale = 1.f;  // FP8 cache
  float v_scale = 1.f;
  ScoreMod mod;
};

// Tensor-core (tcgen05 + TMEM + TMA) path; requires head_dim 64 or 128, bf16, and
// for the paged case a block size that is a multiple of 128 or a divisor of
// 128 of at least 8.
bool prefill_tc_supported(const PrefillArgs& a);
int prefill_tc_launch(const PrefillArgs& a, cudaStream_t stream);
// The same kernel with score modifiers (masks; a cap; a distance bias; both),
// and over an FP8 E4M3 cache; every block size.
int prefill_tc_masked_launch(const PrefillArgs& a, cudaStream_t stream);
int prefill_tc_capped_launch(const PrefillArgs& a, cudaStream_t stream);
int prefill_tc_biased_launch(const PrefillArgs& a, cudaStream_t stream);
int prefill_tc_capped_biased_launch(const PrefillArgs& a, cudaStream_t stream);
int prefill_tc_fp8_launch(const PrefillArgs& a, cudaStream_t stream);
// Chunks over a 4-bit cache.
int prefill_tc_q4_launch(const PrefillArgs& a, cudaStream_t stream);
// Those of at most 8 rows per KV head and 8 KV heads on the decode kernel, with a
// workspace of chunk_decode_workspace_bytes.
int chunk_decode_q4_launch(const PrefillArgs& a, cudaStream_t stream);
// Chunks of at most 8 rows per KV head (max_seqlen_q * G <= 8) on the decode
// kernel; workspace bytes it needs on the current device (0: an error).
int chunk_decode_launch(const PrefillArgs& a, bool fp8, cudaStream_t stream);
size_t chunk_decode_workspace_bytes(int batch, int num_kv_heads, int head_dim);
// Parts a long pair of query tiles may run as, and the bytes of each of the
// split's two counter arrays.
int prefill_tc_parts(int batch, int num_kv_heads, int group, int max_seqlen_q, int sms);
size_t prefill_tc_flag_bytes(long long items);
// Workspace bytes that let the tcgen05 path split long items (0: never splits).
size_t prefill_tc_workspace_bytes(int batch, int num_kv_heads, int group, int head_dim, int max_seqlen_q);

}  // namespace pkv
