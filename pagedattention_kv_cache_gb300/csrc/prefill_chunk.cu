// paged_varlen_prefill_attn_mod and paged_varlen_prefill_attn_fp8: a chunk of
// new tokens per sequence over its keys, with modified scores, or over an
// FP8 E4M3 cache.
//
// Row r of sequence i sits at p = nk - nq + r.  For query head h (KV head
// h / G) and every key t that the row sees,
//     s_t = scale q . K_t;  s_t = c tanh(s_t / c);  s_t -= slope_h |p - t|
//     out = sum_t softmax(s)_t V_t,
// zeros when it sees none.  The row sees first_keys[row] <= t < nk with t <= p
// (causal) or t < prefix_lens[i].
#include <cfloat>

#include "prefill_args.cuh"
#include "score_mod.cuh"

namespace {

using pkv::PrefillArgs;

// Argument checks of both entry points: PKV_OK when a launch may follow, 1
// when there is nothing to do, else the negative status to return.
int check_args(const PrefillArgs& a, int max_seqlen_k) {
  if (a.batch < 0 || a.total_q < 0 || a.total_k < 0 || a.hq <= 0 || a.hkv <= 0 || a.head_dim <= 0 ||
      a.max_seqlen_q < 0 || max_seqlen_k < 0)
    return PKV_EINVAL;
  if (a.hq % a.hkv != 0) return PKV_EINVAL;
  if (a.head_dim != 128 && a.head_dim != 64) return PKV_EUNSUPPORTED;
  if (a.group != 1 && a.group != 2 && a.group != 4 && a.group != 8) return PKV_EUNSUPPORTED;
  if (a.causal != 0 && a.causal != 1) return PKV_EINVAL;
  if (!(a.scale >= FLT_MIN) || isinf(a.scale)) return PKV_EINVAL;
  if (a.batch == 0 || a.max_seqlen_q == 0 || a.total_q == 0) return 1;
  if (!a.out || !a.q || !a.cu_q || !a.cu_k) return PKV_EINVAL;
  if (a.block_tables) {
    if (!a.k_cache || !a.v_cache || a.block_size <= 0 || a.num_blocks <= 0 || a.max_blocks < 0) return PKV_EINVAL;
    if (static_cast<long long>(a.max_blocks) * a.block_size > INT32_MAX ||
        static_cast<long long>(a.num_blocks) * a.block_size > INT32_MAX)
      return PKV_EINVAL;
    if (!pkv::aligned16(a.k_cache) || !pkv::aligned16(a.v_cache)) return PKV_EALIGN;
  } else {
    if (!a.k || !a.v || a.total_k == 0) return PKV_EINVAL;
    if (!pkv::aligned16(a.k) || !pkv::aligned16(a.v)) return PKV_EALIGN;
  }
  if (!pkv::aligned16(a.out) || !pkv::aligned16(a.q)) return PKV_EALIGN;
  if (a.workspace && (reinterpret_cast<uintptr_t>(a.workspace) & 255)) return PKV_EALIGN;
  return PKV_OK;
}

// Whether the decode kernel takes a chunk: at most 8 rows per KV head (its own
// limits are head_dim 128 and 8 KV heads), and work enough.  The tcgen05 kernel
// needs about 6 us and 1 us per 128 keys for each wave of one (sequence, KV head)
// per SM; the decode kernel 8 us, the time of the bytes, and up to 17 us of
// merging, more with more rows.  Measured with 8 KV heads, G = 2, E4M3 (us,
// decode / tcgen05): 4 tokens x 1 sequence after 512 keys 16.9 / 13.8, after
// 2048 21.0 / 25.2; x 16 sequences 27.6 / 14.5 and 30.2 / 35.6; 1 token x 1
// sequence after 128 keys 8.3 / 8.9, after 512 10.2 / 13.8; two waves (64
// sequences) 16.9 / 28.3 after 32 keys.  bf16 moves twice the bytes: 2 tokens x 1
// sequence after 1024 keys 13.0 / 15.9, after 8192 18.7 / 32.5 (E4M3 13.3 / 16.8 and
// 17.8 / 34.3); x 64 after 512 28.0 / 47.0 (23.6 / 50.7).  Fewer KV heads, 2 of
// them with G = 4, 1 token: x 1 after 1024 bf16 11.0 / 15.6, x 16 after 8192 32.6 / 85.3.
// The rule looks at the rows, not at the number of sequences within a wave, and
// is on the wrong side just past its border where several share it: 2 tokens
// x 16 sequences after 512 keys 20.7 / 13.7 (bf16 20.1 / 12.2), after 1024 22.9 / 19.2
// (24.0 / 17.1), bf16 after 2048 30.9 / 27.9 and after 8192 89.0 / 87.2; 2 KV heads,
// G = 4, 1 token x 64 after 2048 bf16 30.9 / 27.9 (E4M3 23.4 / 30.1).
bool short_chunk(int batch, int group, int num_kv_heads, int head_dim, int max_seqlen_q, int max_seqlen_k) {
  const long long rows = static_cast<long long>(max_seqlen_q) * group;
  if (head_dim != 128 || num_kv_heads > 8 || rows > 8) return false;
  pkv::DeviceInfo info;
  if (pkv::device_info(&info) != PKV_OK) return false;
  const bool one_wave = static_cast<long long>(batch) * num_kv_heads <= info.sms;
  return !one_wave || max_seqlen_k > 128 * rows;
}

// The decode kernel runs a short chunk when its workspace is there, else the
// tcgen05 kernel does.
bool on_decode_kernel(const PrefillArgs& a, int max_seqlen_k) {
  if (!a.block_tables || !short_chunk(a.batch, a.group, a.hkv, a.head_dim, a.max_seqlen_q, max_seqlen_k)) return false;
  const size_t need = pkv::chunk_decode_workspace_bytes(a.batch, a.hkv, a.head_dim);
  return need > 0 && a.workspace && a.workspace_bytes >= need;
}

}  // namespace

extern "C" size_t pkv_paged_short_chunk_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                                        int32_t head_dim, int32_t max_seqlen_q,
                                                        int32_t max_seqlen_k) {
  if (batch <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 || max_seqlen_q <= 0)
    return 0;
  const int group = num_q_heads / num_kv_heads;
  if ((group != 1 && group != 2 && group != 4 && group != 8) ||
      !short_chunk(batch, group, num_kv_heads, head_dim, max_seqlen_q, max_seqlen_k))
    return 0;
  return pkv::chunk_decode_workspace_bytes(batch, num_kv_heads, head_dim);
}

extern "C" int pkv_paged_varlen_prefill_attn_mod(
    void* out, const void* q, const void* k, const void* v, const void* k_cache, const void* v_cache,
    const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
    const int32_t* block_tables, int32_t max_blocks_per_seq, int32_t batch, int32_t total_q, int32_t total_k,
    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
    int32_t causal, float softcap, const float* alibi_slopes, const int32_t* first_keys, const int32_t* prefix_lens,
    void* workspace, size_t workspace_bytes, pkv_dtype dtype, pkv_stream_t stream) {
  if (dtype != PKV_BF16) return PKV_EUNSUPPORTED;
  if (!pkv::softcap_valid(softcap) || (prefix_lens && causal != 1)) return PKV_EINVAL;
  PrefillArgs a{};
  a.out = out;
  a.q = q;
  a.k = k;
  a.v = v;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.block_tables = block_tables;
  a.total_q = total_q;
  a.total_k = block_tables ? 0 : total_k;
  a.max_seqlen_q = max_seqlen_q;
  a.max_blocks = max_blocks_per_seq;
  a.batch = batch;
  a.hq = num_q_heads;
  a.hkv = num_kv_heads;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.scale = scale;
  a.causal = causal;
  a.group = num_kv_heads > 0 ? num_q_heads / num_kv_heads : 0;
  a.head_dim = head_dim;
  a.workspace = workspace;
  a.workspace_bytes = workspace ? workspace_bytes : 0;
  a.mod = pkv::make_score_mod(scale, softcap, alibi_slopes, first_keys, prefix_lens);
  const int chk = check_args(a, max_seqlen_k);
  if (chk != PKV_OK) return chk > 0 ? PKV_OK : chk;
  int st = PKV_OK;
  a.err = pkv::device_error_word(&st);
  if (st != PKV_OK) return st;
  if (on_decode_kernel(a, max_seqlen_k)) return pkv::chunk_decode_launch(a, false, stream);
  if (a.mod.slopes)
    return softcap > 0.f || !pkv::raw_bias_scale(scale) ? pkv::prefill_tc_capped_biased_launch(a, stream)
                                                        : pkv::prefill_tc_biased_launch(a, stream);
  return softcap > 0.f ? pkv::prefill_tc_capped_launch(a, stream) : pkv::prefill_tc_masked_launch(a, stream);
}

extern "C" int pkv_paged_varlen_prefill_attn_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                                                 const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                                                 int32_t max_seqlen_q, int32_t max_seqlen_k,
                                                 const int32_t* block_tables, int32_t max_blocks_per_seq,
                                                 int32_t batch, int32_t total_q, int32_t num_q_heads,
                                                 int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                                 int32_t num_blocks, float scale, float k_scale, float v_scale,
                                                 int32_t causal, void* workspace, size_t workspace_bytes,
                                                 pkv_stream_t stream) {
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || isinf(k_scale) || isinf(v_scale)) return PKV_EINVAL;
  PrefillArgs a{};
  a.out = out;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.block_tables = block_tables;
  a.total_q = total_q;
  a.max_seqlen_q = max_seqlen_q;
  a.max_blocks = max_blocks_per_seq;
  a.batch = batch;
  a.hq = num_q_heads;
  a.hkv = num_kv_heads;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.scale = scale;
  a.causal = causal;
  a.group = num_kv_heads > 0 ? num_q_heads / num_kv_heads : 0;
  a.head_dim = head_dim;
  a.workspace = workspace;
  a.workspace_bytes = workspace ? workspace_bytes : 0;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const int chk = check_args(a, max_seqlen_k);
  if (chk != PKV_OK) return chk > 0 ? PKV_OK : chk;
  if (!block_tables) return PKV_EINVAL;
  int st = PKV_OK;
  a.err = pkv::device_error_word(&st);
  if (st != PKV_OK) return st;
  if (on_decode_kernel(a, max_seqlen_k)) return pkv::chunk_decode_launch(a, true, stream);
  return pkv::prefill_tc_fp8_launch(a, stream);
}
