// Chunks of a few new tokens per sequence (at most 8 rows per KV head: drafted
// tokens to be checked, the last tokens of a prompt) on the decode kernel of
// decode_mma.cuh, bf16 with score modifiers or an FP8 E4M3 cache.
//
// Such a chunk reads every key for a handful of rows, so it is bound by HBM as
// decode is.  The tcgen05 prefill pads its rows to tiles of 128 and walks a
// sequence's keys in one CTA per KV head; the decode kernel divides the batch's
// keys evenly over the SMs and streams all KV heads of a key at once.
#include "decode_launch.cuh"
#include "prefill_args.cuh"

namespace {

constexpr int kChunkRows = 8;  // G * QL of every instantiation

template <typename TC, bool kMod>
int dispatch_chunk(Params& p, int group, int sms, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_mma<1, kChunkRows, TC, kMod, true>(p, sms, stream);
    case 2: return launch_mma<2, kChunkRows / 2, TC, kMod, true>(p, sms, stream);
    case 4: return launch_mma<4, kChunkRows / 4, TC, kMod, true>(p, sms, stream);
    default: return launch_mma<8, kChunkRows / 8, TC, kMod, true>(p, sms, stream);
  }
}

}  // namespace

namespace pkv {

size_t chunk_decode_workspace_bytes(int batch, int num_kv_heads, int head_dim) {
  DeviceInfo info;
  if (device_info(&info) != PKV_OK) return 0;
  size_t a, b;
  return workspace_layout(batch, kChunkRows * num_kv_heads, head_dim, 0, info.sms, &a, &b);
}

int chunk_decode_launch(const PrefillArgs& a, bool fp8, cudaStream_t stream) {
  DeviceInfo info;
  if (device_info(&info) != PKV_OK) return PKV_ECUDA;
  Params p{};
  size_t off_o = 0, off_ml = 0;
  const size_t need = workspace_layout(a.batch, kChunkRows * a.hkv, a.head_dim, 0, info.sms, &off_o, &off_ml);
  if (!a.workspace || a.workspace_bytes < need) return PKV_EWORKSPACE;
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  p.counters = reinterpret_cast<int32_t*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + off_o);
  p.part_ml = reinterpret_cast<float*>(ws + off_ml);
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
  p.scale_log2 = a.scale * kLog2e * (fp8 ? a.k_scale : 1.f);
  p.v_scale = fp8 ? a.v_scale : 1.f;
  p.mod = a.mod;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.total_q = a.total_q;
  p.max_seqlen_q = a.max_seqlen_q;
  p.causal = a.causal;
  return fp8 ? dispatch_chunk<__nv_fp8_e4m3, false>(p, a.group, info.sms, stream)
             : dispatch_chunk<__nv_bfloat16, true>(p, a.group, info.sms, stream);
}

}  // namespace pkv
