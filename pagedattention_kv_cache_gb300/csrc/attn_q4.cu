// Attention over the 4-bit cache, one warp per (query row, query head): the
// entry point paged_decode_attn_q4 and the kernel that
// paged_varlen_prefill_attn_q4 (prefill_chunk.cu) launches too.
//
// s_t = scale q . K_t, out = sum_t softmax(s)_t V_t over the keys the row sees,
// K_t and V_t the values that the cache stands for (q4.cuh).
#include <cmath>

#include "prefill_args.cuh"
#include "q4.cuh"

namespace {

struct Q4Params {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const unsigned char* k_cache;
  const unsigned char* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;  // decode; null: chunks by cu_q / cu_k
  const int32_t* cu_q;
  const int32_t* cu_k;
  unsigned int* err;
  int max_blocks, total_q, max_seqlen_q, hq, hkv, block_size, num_blocks, causal;
  float scale_log2, v_scale;
};

template <int D>
__global__ void __launch_bounds__(128) attn_q4_kernel(const Q4Params p) {
  pkv::pdl_enter();
  constexpr int EPL = D / 32;  // elements per lane
  const int seq = blockIdx.y;
  const int lane = threadIdx.x % 32;
  const int item = blockIdx.x * 4 + threadIdx.x / 32;
  const int r = item / p.hq, h = item - r * p.hq;
  int q0 = seq, nq = 1, nk = 0;
  bool bad;
  if (p.context_lens) {
    nk = __ldg(p.context_lens + seq);
    bad = nk < 0;
  } else {
    q0 = __ldg(p.cu_q + seq);
    nq = __ldg(p.cu_q + seq + 1) - q0;
    nk = __ldg(p.cu_k + seq + 1) - __ldg(p.cu_k + seq);
    bad = q0 < 0 || nq < 0 || nk < nq || static_cast<long long>(q0) + nq > p.total_q || nq > p.max_seqlen_q;
  }
  if (bad || nk > static_cast<long long>(p.max_blocks) * p.block_size) {
    if (threadIdx.x == 0) pkv::raise_error(p.err, PKV_DERR_LEN_RANGE);
    if (!p.context_lens) return;
    nk = 0;
  }
  if (r >= nq) return;
  const int g = h / (p.hq / p.hkv);
  const size_t at = (static_cast<size_t>(q0 + r) * p.hq + h) * D + lane * EPL;
  float q[EPL], acc[EPL] = {};
#pragma unroll
  for (int e = 0; e < EPL; ++e) q[e] = __bfloat162float(p.q[at + e]) * p.scale_log2;
  const size_t row_bytes = pkv::q4_row_bytes(p.hkv, D);
  const int code_at = g * (D / 2) + lane * (EPL / 2);
  const int scale_at = pkv::q4_scale_offset(p.hkv, D) + (g * D + lane * EPL) / 16;
  const int end = p.context_lens || !p.causal ? nk : nk - nq + r + 1;
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < end; ++t) {
    const int block = __ldg(p.block_tables + static_cast<size_t>(seq) * p.max_blocks + t / p.block_size);
    if (block < 0 || block >= p.num_blocks) {
      if (lane == 0) pkv::raise_error(p.err, PKV_DERR_BLOCK_RANGE);
      continue;
    }
    const size_t row = (static_cast<size_t>(block) * p.block_size + t % p.block_size) * row_bytes;
    const float ks = pkv::e4m3_value(p.k_cache[row + scale_at]), vs = pkv::e4m3_value(p.v_cache[row + scale_at]);
    float s = 0.f, v[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      const int kc = p.k_cache[row + code_at + e / 2] >> (4 * (e & 1)) & 15;
      const int vc = p.v_cache[row + code_at + e / 2] >> (4 * (e & 1)) & 15;
      s = fmaf(q[e], static_cast<float>(kc - 8) * ks, s);
      v[e] = static_cast<float>(vc - 8) * vs;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float mn = pkv::max_keep_nan(m, s);
    const float keep = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float w = mn == -INFINITY ? 0.f : exp2f(s - mn);
    l = fmaf(l, keep, w);
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = fmaf(acc[e], keep, w * v[e]);
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : p.v_scale / l;
#pragma unroll
  for (int e = 0; e < EPL; ++e) p.out[at + e] = __float2bfloat16_rn(acc[e] * inv);
}

int launch_q4(const Q4Params& p, int batch, int head_dim, cudaStream_t stream) {
  const dim3 grid((static_cast<unsigned>(p.max_seqlen_q) * p.hq + 3) / 4, batch);
  const cudaError_t e = head_dim == 64 ? pkv::launch_pdl(attn_q4_kernel<64>, grid, dim3(128), 0, stream, p)
                                       : pkv::launch_pdl(attn_q4_kernel<128>, grid, dim3(128), 0, stream, p);
  return e == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

}  // namespace

namespace pkv {

int chunk_q4_launch(const PrefillArgs& a, cudaStream_t stream) {
  const Q4Params p{static_cast<__nv_bfloat16*>(a.out), static_cast<const __nv_bfloat16*>(a.q),
                   static_cast<const unsigned char*>(a.k_cache), static_cast<const unsigned char*>(a.v_cache),
                   a.block_tables, nullptr, a.cu_q, a.cu_k, a.err, a.max_blocks, a.total_q, a.max_seqlen_q, a.hq, a.hkv,
                   a.block_size, a.num_blocks, a.causal, a.scale * kLog2e * a.k_scale, a.v_scale};
  return launch_q4(p, a.batch, a.head_dim, stream);
}

}  // namespace pkv

extern "C" int pkv_paged_decode_attn_q4(void* out, const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                                        const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                        int32_t num_blocks, float scale, float k_scale, float v_scale,
                                        int32_t num_splits, void* workspace, size_t workspace_bytes,
                                        pkv_stream_t stream) {
  if (batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      num_blocks < 0 || max_blocks_per_seq < 0 || num_splits < 0)
    return PKV_EINVAL;
  if (num_q_heads % num_kv_heads != 0) return PKV_EINVAL;
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || std::isinf(k_scale) || std::isinf(v_scale)) return PKV_EINVAL;
  if (!pkv::q4_head_dim(head_dim) || num_kv_heads > 8) return PKV_EUNSUPPORTED;
  const int group = num_q_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_EUNSUPPORTED;
  if (static_cast<long long>(max_blocks_per_seq) * block_size > INT32_MAX) return PKV_EINVAL;
  if (batch == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PKV_EINVAL;
  if (!pkv::aligned16(out) || !pkv::aligned16(q) || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache))
    return PKV_EALIGN;
  int st = PKV_OK;
  unsigned int* err = pkv::device_error_word(&st);
  if (st != PKV_OK) return st;
  Q4Params p{};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const unsigned char*>(k_cache);
  p.v_cache = static_cast<const unsigned char*>(v_cache);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.err = err;
  p.max_blocks = max_blocks_per_seq;
  p.max_seqlen_q = 1;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * pkv::kLog2e * k_scale;
  p.v_scale = v_scale;
  return launch_q4(p, batch, head_dim, stream);
}
