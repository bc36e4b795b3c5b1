// paged_decode_attn_q4, and short chunks of paged_varlen_prefill_attn_q4, on the
// kernel of decode_q4.cuh.
//
// out = sum_t softmax(scale q . K_t) V_t over t < context_lens[b] (zeros for an
// empty context), K_t and V_t the values the 4-bit rows stand for.
#include "decode_launch.cuh"
#include "decode_q4_args.cuh"
#include "prefill_args.cuh"
#include "q4.cuh"

namespace pkv {

int chunk_decode_q4_launch(const PrefillArgs& a, cudaStream_t stream) {
  Q4Decode d{};
  d.out = a.out;
  d.q = a.q;
  d.k_cache = a.k_cache;
  d.v_cache = a.v_cache;
  d.block_tables = a.block_tables;
  d.cu_q = a.cu_q;
  d.cu_k = a.cu_k;
  d.err = a.err;
  d.max_blocks = a.max_blocks;
  d.batch = a.batch;
  d.hq = a.hq;
  d.hkv = a.hkv;
  d.block_size = a.block_size;
  d.num_blocks = a.num_blocks;
  d.total_q = a.total_q;
  d.max_seqlen_q = a.max_seqlen_q;
  d.causal = a.causal;
  d.scale = a.scale;
  d.k_scale = a.k_scale;
  d.v_scale = a.v_scale;
  d.workspace = a.workspace;
  d.workspace_bytes = a.workspace_bytes;
  return a.head_dim == 64 ? decode_q4_d64(d, stream) : decode_q4_d128(d, stream);
}

}  // namespace pkv

extern "C" int pkv_paged_decode_attn_q4(void* out, const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                                        const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                        int32_t num_blocks, float scale, float k_scale, float v_scale,
                                        int32_t num_splits, void* workspace, size_t workspace_bytes,
                                        pkv_stream_t stream) {
  if (!pkv::q4_attention_scale(k_scale) || !pkv::q4_attention_scale(v_scale)) return PKV_EINVAL;
  const int chk = check_decode_args(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, batch,
                                    num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, num_splits, PKV_BF16);
  if (chk < 0) return chk;
  const int group = num_q_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_EUNSUPPORTED;
  if (chk > 0) return PKV_OK;
  int st = PKV_OK;
  unsigned int* err = pkv::device_error_word(&st);
  if (st != PKV_OK) return st;
  pkv::Q4Decode d{};
  d.out = out;
  d.q = q;
  d.k_cache = k_cache;
  d.v_cache = v_cache;
  d.block_tables = block_tables;
  d.context_lens = context_lens;
  d.err = err;
  d.max_blocks = max_blocks_per_seq;
  d.batch = batch;
  d.hq = num_q_heads;
  d.hkv = num_kv_heads;
  d.block_size = block_size;
  d.num_blocks = num_blocks;
  d.scale = scale;
  d.k_scale = k_scale;
  d.v_scale = v_scale;
  d.num_splits = num_splits;
  d.workspace = workspace;
  d.workspace_bytes = workspace_bytes;
  return head_dim == 64 ? pkv::decode_q4_d64(d, stream) : pkv::decode_q4_d128(d, stream);
}
