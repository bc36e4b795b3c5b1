// paged_decode_attn_mod: decode with modified scores (softcap, distance bias,
// first visible key), on the kernels of decode_mma.cuh and decode_simt.cuh
// instantiated with kMod.
//
// For sequence b of length T with the query at p = T - 1 and head h:
//     s_t = scale q . K_t;  s_t = c tanh(s_t / c);  s_t -= slope_h (p - t)
//     out = sum_{first_b <= t < T} softmax(s)_t V_t     (zeros when no t is left)
// Bound: HBM, the visible K / V rows once.  The split plan counts visible
// tokens only (from first_b, down to the 16-token box that holds it), so a
// window of W keys costs what a context of W tokens costs, however long the
// context is.
#include "decode_launch.cuh"

extern "C" int pkv_paged_decode_attn_mod(void* out, const void* q, const void* k_cache, const void* v_cache,
                                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                                         const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
                                         int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                         int32_t num_blocks, float scale, float softcap, const float* alibi_slopes,
                                         const int32_t* first_keys, int32_t num_splits, void* workspace,
                                         size_t workspace_bytes, pkv_dtype dtype, pkv_stream_t stream) {
  if (!pkv::softcap_valid(softcap)) return PKV_EINVAL;
  const int chk = check_decode_args(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, batch,
                                    num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, num_splits, dtype);
  if (chk != PKV_OK) return chk > 0 ? PKV_OK : chk;
  return run_decode<true>(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, batch, num_q_heads,
                          num_kv_heads, head_dim, block_size, num_blocks, scale,
                          pkv::make_score_mod(scale, softcap, alibi_slopes, first_keys, nullptr), num_splits, workspace,
                          workspace_bytes, dtype, stream);
}
