// Attention of chunks over the 4-bit cache (paged_varlen_prefill_attn_q4), one warp
// per (query row, query head).
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
  const int q0 = __ldg(p.cu_q + seq), nq = __ldg(p.cu_q + seq + 1) - q0;
  const int nk = __ldg(p.cu_k + seq + 1) - __ldg(p.cu_k + seq);
  if (q0 < 0 || nq < 0 || nk < nq || static_cast<long long>(q0) + nq > p.total_q || nq > p.max_seqlen_q ||
      nk > static_cast<long long>(p.max_blocks) * p.block_size) {
    if (threadIdx.x == 0) pkv::raise_error(p.err, PKV_DERR_LEN_RANGE);
    return;
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
  const int end = !p.causal ? nk : nk - nq + r + 1;
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
                   a.block_tables, a.cu_q, a.cu_k, a.err, a.max_blocks, a.total_q, a.max_seqlen_q, a.hq, a.hkv,
                   a.block_size, a.num_blocks, a.causal, a.scale * kLog2e * a.k_scale, a.v_scale};
  return launch_q4(p, a.batch, a.head_dim, stream);
}

}  // namespace pkv
