// paged_decode_attn_q4, and short chunks of paged_varlen_prefill_attn_q4, on the
// kernel of decode_q4.cuh.
//
// out = sum_t softmax(scale q . K_t) V_t over t < context_lens[b] (zeros for an
// empty context), K_t and V_t the values the 4-bit rows stand for.
#include "decode_launch.cuh"
#include "decode_q4.cuh"
#include "prefill_args.cuh"

namespace {

constexpr int kChunkRows = 8;  // G * QL of the chunk instantiations

template <int D, bool kVar>
int dispatch_q4(Params& p, int group, int sms, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_q4<1, kVar ? kChunkRows : 1, D, kVar>(p, sms, stream);
    case 2: return launch_q4<2, kVar ? kChunkRows / 2 : 1, D, kVar>(p, sms, stream);
    case 4: return launch_q4<4, kVar ? kChunkRows / 4 : 1, D, kVar>(p, sms, stream);
    default: return launch_q4<8, 1, D, kVar>(p, sms, stream);
  }
}

// Points p at the parts of a split workspace of `rows` query rows per sequence.
int take_workspace(Params& p, void* workspace, size_t workspace_bytes, int batch, int rows, int head_dim, int num_splits,
                   int sms) {
  size_t off_o = 0, off_ml = 0;
  const size_t need = workspace_layout(batch, rows, head_dim, num_splits, sms, &off_o, &off_ml);
  if (need == 0) return PKV_OK;
  if (!workspace || workspace_bytes < need) return PKV_EWORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PKV_EALIGN;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.counters = reinterpret_cast<int32_t*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + off_o);
  p.part_ml = reinterpret_cast<float*>(ws + off_ml);
  return PKV_OK;
}

}  // namespace

namespace pkv {

int chunk_decode_q4_launch(const PrefillArgs& a, cudaStream_t stream) {
  DeviceInfo info;
  if (device_info(&info) != PKV_OK) return PKV_ECUDA;
  Params p{};
  const int st = take_workspace(p, a.workspace, a.workspace_bytes, a.batch, kChunkRows * a.hkv, a.head_dim, 0, info.sms);
  if (st != PKV_OK) return st;
  p.out = a.out;
  p.q = a.q;
  p.k_cache = static_cast<const unsigned char*>(a.k_cache);
  p.v_cache = static_cast<const unsigned char*>(a.v_cache);
  p.block_tables = a.block_tables;
  p.err = a.err;
  p.max_blocks = a.max_blocks;
  p.batch = a.batch;
  p.hq = a.hq;
  p.ql = 1;
  p.hkv = a.hkv;
  p.block_size = a.block_size;
  p.num_blocks = a.num_blocks;
  p.scale_log2 = a.scale * kLog2e * a.k_scale;
  p.v_scale = a.v_scale;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.total_q = a.total_q;
  p.max_seqlen_q = a.max_seqlen_q;
  p.causal = a.causal;
  return a.head_dim == 64 ? dispatch_q4<64, true>(p, a.group, info.sms, stream)
                          : dispatch_q4<128, true>(p, a.group, info.sms, stream);
}

}  // namespace pkv

extern "C" int pkv_paged_decode_attn_q4(void* out, const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                                        const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                        int32_t num_blocks, float scale, float k_scale, float v_scale,
                                        int32_t num_splits, void* workspace, size_t workspace_bytes,
                                        pkv_stream_t stream) {
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || isinf(k_scale) || isinf(v_scale)) return PKV_EINVAL;
  const int chk = check_decode_args(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, batch,
                                    num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, num_splits, PKV_BF16);
  if (chk < 0) return chk;
  const int group = num_q_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_EUNSUPPORTED;
  if (chk > 0) return PKV_OK;
  pkv::DeviceInfo info;
  if (pkv::device_info(&info) != PKV_OK) return PKV_ECUDA;
  int st = PKV_OK;
  unsigned int* err = pkv::device_error_word(&st);
  if (st != PKV_OK) return st;
  Params p{};
  st = take_workspace(p, workspace, workspace_bytes, batch, num_q_heads, head_dim, num_splits, info.sms);
  if (st != PKV_OK) return st;
  p.out = out;
  p.q = q;
  p.k_cache = static_cast<const unsigned char*>(k_cache);
  p.v_cache = static_cast<const unsigned char*>(v_cache);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.err = err;
  p.max_blocks = max_blocks_per_seq;
  p.batch = batch;
  p.hq = num_q_heads;
  p.ql = 1;
  p.hkv = num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * pkv::kLog2e * k_scale;
  p.v_scale = v_scale;
  p.num_splits = num_splits;
  return head_dim == 64 ? dispatch_q4<64, false>(p, group, info.sms, stream)
                        : dispatch_q4<128, false>(p, group, info.sms, stream);
}
