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
#include "prefill_args.cuh"
#include "score_mod.cuh"

namespace {

using pkv::PrefillArgs;

// One warp per (query row, query head): lanes split head_dim, keys one at a
// time with an online softmax in fp32.
template <int D, bool kFp8>
__global__ void __launch_bounds__(128) prefill_rows_kernel(const PrefillArgs a) {
  pkv::pdl_enter();
  constexpr int E = D / 32;
  const int seq = blockIdx.y;
  const int h = blockIdx.z;
  const int g = h / a.group;
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int q_begin = __ldg(a.cu_q + seq);
  const int nq = __ldg(a.cu_q + seq + 1) - q_begin;
  const int k_begin = __ldg(a.cu_k + seq);
  const int nk = __ldg(a.cu_k + seq + 1) - k_begin;
  if (q_begin < 0 || nq < 0 || nk < nq || static_cast<long long>(q_begin) + nq > a.total_q || nq > a.max_seqlen_q ||
      (a.block_tables ? static_cast<long long>(nk) > static_cast<long long>(a.max_blocks) * a.block_size
                      : (k_begin < 0 || static_cast<long long>(k_begin) + nk > a.total_k))) {
    if (threadIdx.x == 0) pkv::raise_error(a.err, PKV_DERR_LEN_RANGE);
    return;
  }
  const int r = blockIdx.x * 4 + warp;
  if (r >= nq) return;
  const int row = q_begin + r;
  const int pos = nk - nq + r;
  int lo = 0, hi = a.causal ? pos + 1 : nk;
  if (a.mod.first_keys) lo = max(0, __ldg(a.mod.first_keys + row));
  if (a.mod.prefix_lens) hi = max(hi, min(__ldg(a.mod.prefix_lens + seq), nk));
  const float slope = a.mod.slopes ? __ldg(a.mod.slopes + h) * pkv::kLog2e : 0.f;
  const float k_mul = kFp8 ? a.k_scale : 1.f;
  float q[E], o[E];
  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<size_t>(row) * a.hq + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qp[e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  auto load = [&](const void* base, size_t at, float* f) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (kFp8)
        f[e] = static_cast<float>(static_cast<const __nv_fp8_e4m3*>(base)[at + e]);
      else
        f[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at + e]);
    }
  };
  for (int t = lo; t < hi; ++t) {
    size_t token;
    if (a.block_tables) {
      const int phys = __ldg(a.block_tables + static_cast<size_t>(seq) * a.max_blocks + t / a.block_size);
      if (phys < 0 || phys >= a.num_blocks) {
        pkv::raise_error(a.err, PKV_DERR_BLOCK_RANGE);
        continue;
      }
      token = static_cast<size_t>(phys) * a.block_size + t % a.block_size;
    } else {
      token = static_cast<size_t>(k_begin) + t;
    }
    const size_t at = (token * a.hkv + g) * D + lane * E;
    float k[E], v[E];
    load(a.block_tables ? a.k_cache : a.k, at, k);
    load(a.block_tables ? a.v_cache : a.v, at, v);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    float x = s * (a.scale * k_mul * pkv::kLog2e);
    if (a.mod.cap_log2 > 0.f) x = a.mod.cap_log2 * tanhf(s * a.mod.raw_to_x);
    x = fmaf(-slope, fabsf(static_cast<float>(pos - t)), x);
    const float mn = fmaxf(m, x);
    if (mn == -INFINITY) continue;
    const float c = exp2f(m - mn);
    const float w = exp2f(x - mn);
    l = fmaf(l, c, w);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], c, w * v[e]);
    m = mn;
  }
  const float inv = l > 0.f ? (kFp8 ? a.v_scale : 1.f) / l : 0.f;
  __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) + (static_cast<size_t>(row) * a.hq + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) op[e] = __float2bfloat16_rn(o[e] * inv);
}

int launch_rows(const PrefillArgs& a, bool fp8, cudaStream_t stream) {
  const dim3 grid((a.max_seqlen_q + 3) / 4, a.batch, a.hq);
  auto kernel = a.head_dim == 64 ? (fp8 ? prefill_rows_kernel<64, true> : prefill_rows_kernel<64, false>)
                                 : (fp8 ? prefill_rows_kernel<128, true> : prefill_rows_kernel<128, false>);
  return pkv::launch_pdl(kernel, grid, dim3(128), 0, stream, a) == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

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
  if (!(a.scale > 0.f) || isinf(a.scale)) return PKV_EINVAL;
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

}  // namespace

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
  return pkv::prefill_tc_mod_launch(a, stream);
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
  return launch_rows(a, true, stream);
}
