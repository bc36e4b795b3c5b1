// Paged decode / verify attention kernel shared by the decode entry points
// (one query token per sequence, decode.cu) and the verify entry point (QL
// query tokens per sequence, verify.cu).
//
//
// What is computed ("3.6 ModelRunner, CUDA Graph, and benchmarks", section 2,
// decode; section 5, padding rows): for sequence b and query head h reading
// KV head g = h / G, over t < context_lens[b],
//     s_t = scale * q[b, h] . K_t,  out[b, h] = sum_t softmax(s)_t V_t,
// with K_t / V_t at physical block block_tables[b, t / bs], offset t % bs.
// context_lens 0 writes zeros and reads nothing.
//
// How (GB300 design), shared by both kernels:
//  * A CTA covers every KV head of a token range, so each token's K (or V)
//    row of all heads, [Hkv, D], is contiguous in the [blocks, bs, Hkv, D]
//    pool.  A producer warp streams the range into a ring of shared-memory
//    stages with TMA copies completed on mbarriers; every K/V byte is read from
//    HBM once, and all G query heads of a KV head reuse it on chip.
//  * Consumer warps, one per (KV head, token phase), fold each stage into a
//    running online softmax (exp2 domain) and accumulate P.V.
//  * Split over the context: the batch's context tokens, flattened, are
//    divided evenly over the grid (automatic mode) or each sequence into S
//    equal parts.  A sequence covered by one CTA is written directly; otherwise
//    each part writes (o, m, l) to the workspace and atomic tickets (no
//    waiting) elect the CTAs that merge the parts by log-sum-exp.
// paged_decode_mma_kernel (mma.sync tensor cores, 16-token tensor copies)
// runs every bf16 or FP8 cache with head_dim 128; paged_decode_kernel (CUDA
// cores, 1-D bulk copies of token spans) runs fp32 caches, and bf16 with head_dim 64.
// Two template switches give both kernels further uses: kMod, score modifiers
// (decode_mod.cu; bf16 with head_dim 64 runs on the tensor cores there), and,
// for the first, kVar, short chunks of new tokens (chunk_decode.cu).
//
// Verify (speculative-decoding target pass, QL > 1): query token i of
// sequence b sits at position context_lens[b] - QL + i and attends keys up to
// it, so the QL tokens just stored are causally masked among themselves.  The
// warp's rows become (query token, head) pairs; K/V are still read once.
//
// Files: decode_plan.cuh (parameters, split plan, merge), decode_simt.cuh
// and decode_mma.cuh (the two kernels), this file (host side: launch shapes,
// the split workspace layout and the dispatch over group sizes).  The entry
// points that include it are decode.cu, decode_mod.cu, verify.cu, fp8.cu and
// chunk_decode.cu.
#pragma once

#include <algorithm>

#include "decode_mma.cuh"
#include "decode_simt.cuh"

namespace {

// ------------------------------------------------------------------ host side

struct LaunchShape {
  int nw, wph, t_stage, stages;
  size_t stage_bytes, smem;
};

template <typename T, int D, int R>
LaunchShape launch_shape(int hkv) {
  using S = Shape<T, D, R>;
  LaunchShape ls;
  ls.wph = hkv >= 8 ? 1 : 8 / hkv;
  ls.nw = hkv * ls.wph;
  ls.t_stage = S::ROUNDS * S::TPW * ls.wph;
  ls.stage_bytes = static_cast<size_t>(ls.t_stage) * hkv * S::ROW_BYTES * 2;
  const size_t misc = 2 * kMaxStages * sizeof(uint64_t) + 64 * sizeof(long long) + 32 * sizeof(int) +
                      (ls.wph > 1 ? static_cast<size_t>(ls.nw) * R * (D + 2) * sizeof(float) : 0);
  int stages = static_cast<int>((kSmemBudget - misc) / ls.stage_bytes);
  ls.stages = stages > kMaxStages ? kMaxStages : stages;
  ls.smem = ls.stages * ls.stage_bytes + misc;
  return ls;
}

size_t slot_count(int batch, int num_splits, int sms) {
  if (num_splits == 1) return 0;
  if (num_splits > 1) return static_cast<size_t>(batch) * num_splits;
  return static_cast<size_t>(sms) * kWorkspaceCtasPerSm + batch;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

size_t workspace_layout(int batch, int hq, int d, int num_splits, int sms, size_t* off_o, size_t* off_ml) {
  const size_t slots = slot_count(batch, num_splits, sms);
  if (slots == 0) return 0;
  // tickets: one per sequence, then one per slot (the merge groups), in the
  // fixed counter area (larger only past 16,384 counters)
  const size_t counters =
      std::max(pkv::kWorkspaceCounterBytes, align256((static_cast<size_t>(batch) + slots) * sizeof(int32_t)));
  *off_o = counters;
  *off_ml = counters + align256(slots * hq * d * sizeof(float));
  return *off_ml + align256(slots * hq * 2 * sizeof(float));
}

template <typename T, typename TC, int D, int G, int QL, bool kMod = false>
int launch(Params& p, int sms, cudaStream_t stream) {
  const LaunchShape ls = launch_shape<TC, D, G * QL>(p.hkv);
  if (ls.stages < 2) return PKV_EUNSUPPORTED;
  p.nw = ls.nw;
  p.wph = ls.wph;
  p.t_stage = ls.t_stage;
  p.stages = ls.stages;
  p.stage_bytes = ls.stage_bytes;
  auto kernel = paged_decode_kernel<T, TC, D, G, QL, kMod>;
  static std::atomic<uint64_t> smem_allowed{0};  // the limit for every number of KV heads
  if (pkv::allow_smem(kernel, kSmemBudget + 1024, smem_allowed) != cudaSuccess) return PKV_ECUDA;
  unsigned grid;
  if (p.num_splits > 0)
    grid = static_cast<unsigned>(static_cast<long long>(p.batch) * p.num_splits);
  else
    grid = static_cast<unsigned>(sms * kAutoCtasPerSm);
  if (grid == 0) return PKV_OK;
  return pkv::launch_pdl(kernel, dim3(grid), dim3((ls.nw + 1) * 32), ls.smem, stream, p) == cudaSuccess ? PKV_OK
                                                                                                       : PKV_ECUDA;
}

template <int G, int QL, typename TC = __nv_bfloat16, bool kMod = false, bool kVar = false, int D = 128>
int launch_mma(Params& p, int sms, cudaStream_t stream) {
  constexpr int ES = static_cast<int>(sizeof(TC));
  constexpr int R = G * QL;
  LaunchShape ls;
  ls.wph = p.hkv >= 8 ? 1 : 8 / p.hkv;
  ls.nw = p.hkv * ls.wph;
  ls.t_stage = kMmaTokens * mma_chunks_per_warp<TC, D>() * ls.wph;
  // tensor-copy layout when every 16-token box lies in one block
  alignas(64) CUtensorMap maps[2];
  std::memset(maps, 0, sizeof(maps));
  p.tma = (p.block_size % kMmaTokens == 0 && p.num_blocks > 0) ? 1 : 0;
  if (p.tma) {
    if (pkv::encode_paged_kv(&maps[0], p.k_cache, p.block_size, p.hkv, p.num_blocks, ES, D) != PKV_OK ||
        pkv::encode_paged_kv(&maps[1], p.v_cache, p.block_size, p.hkv, p.num_blocks, ES, D) != PKV_OK)
      return PKV_ECUDA;
    p.align = kMmaTokens;
    ls.stage_bytes = static_cast<size_t>(ls.t_stage) * p.hkv * D * ES * 2;
  } else {
    p.align = 1;
    const size_t ts = static_cast<size_t>(p.hkv) * D * ES + kMmaPad;
    ls.stage_bytes = static_cast<size_t>(ls.t_stage) * ts * 2;
  }
  // 1024 bytes of slack put the stages on a swizzle-period boundary
  const size_t misc = 1024 + 2 * kMaxStages * sizeof(uint64_t) + 64 * sizeof(long long) + 32 * sizeof(int) +
                      (ls.wph > 1 ? static_cast<size_t>(ls.nw) * R * (D + 2) * sizeof(float) : 0);
  const int stages = static_cast<int>((kSmemBudget - misc) / ls.stage_bytes);
  ls.stages = stages > kMaxStages ? kMaxStages : stages;
  if (ls.stages < 2) return PKV_EUNSUPPORTED;
  ls.smem = ls.stages * ls.stage_bytes + misc;
  p.nw = ls.nw;
  p.wph = ls.wph;
  p.t_stage = ls.t_stage;
  p.stages = ls.stages;
  p.stage_bytes = ls.stage_bytes;
  auto kernel = paged_decode_mma_kernel<G, QL, TC, kMod, kVar, D>;
  static std::atomic<uint64_t> smem_allowed{0};  // the limit for every number of KV heads
  if (pkv::allow_smem(kernel, kSmemBudget + 1024, smem_allowed) != cudaSuccess) return PKV_ECUDA;
  unsigned grid;
  if (p.num_splits > 0)
    grid = static_cast<unsigned>(static_cast<long long>(p.batch) * p.num_splits);
  else
    grid = static_cast<unsigned>(sms * kAutoCtasPerSm);
  if (grid == 0) return PKV_OK;
  return pkv::launch_pdl(kernel, dim3(grid), dim3((ls.nw + 1) * 32), ls.smem, stream, p, maps[0], maps[1]) ==
                 cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

template <typename T, int D, int G, bool kMod>
int launch_g(Params& p, int sms, cudaStream_t stream) {
  // head_dim 64 with score modifiers runs on the tensor cores too: 24 sequences
  // of about 1800 tokens, 4 KV heads, G = 8, took 70 us on the CUDA cores
  if constexpr (std::is_same<T, __nv_bfloat16>::value && (D == 128 || kMod))
    return launch_mma<G, 1, __nv_bfloat16, kMod, false, D>(p, sms, stream);
  else
    return launch<T, T, D, G, 1, kMod>(p, sms, stream);
}

template <typename T, int D, bool kMod = false>
int dispatch_g(Params& p, int group, int sms, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_g<T, D, 1, kMod>(p, sms, stream);
    case 2: return launch_g<T, D, 2, kMod>(p, sms, stream);
    case 4: return launch_g<T, D, 4, kMod>(p, sms, stream);
    case 8: return launch_g<T, D, 8, kMod>(p, sms, stream);
    default: return PKV_EUNSUPPORTED;
  }
}

// Argument checks shared by the decode entry points (everything but the
// workspace): PKV_OK when a launch may follow, 1 when batch is 0 (nothing to
// do), else the negative status to return.
int check_decode_args(const void* out, const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                      int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                      int32_t block_size, int32_t num_blocks, int32_t num_splits, pkv_dtype dtype) {
  if (batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      num_blocks < 0 || max_blocks_per_seq < 0 || num_splits < 0)
    return PKV_EINVAL;
  if (num_q_heads % num_kv_heads != 0) return PKV_EINVAL;
  if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_EUNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PKV_EUNSUPPORTED;
  if (num_kv_heads > 8) return PKV_EUNSUPPORTED;
  if (static_cast<long long>(max_blocks_per_seq) * block_size > INT32_MAX) return PKV_EINVAL;
  if (batch == 0) return 1;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PKV_EINVAL;
  if (!pkv::aligned16(out) || !pkv::aligned16(q) || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache))
    return PKV_EALIGN;
  return PKV_OK;
}

// Runs decode on arguments that check_decode_args accepted: the workspace
// check, the parameters, and the kernel for the type and head_dim.
template <bool kMod>
int run_decode(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
               int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
               int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
               const pkv::ScoreMod& mod, int32_t num_splits, void* workspace, size_t workspace_bytes,
               pkv_dtype dtype, cudaStream_t stream) {
  pkv::DeviceInfo info;
  if (pkv::device_info(&info) != PKV_OK) return PKV_ECUDA;
  int st = PKV_OK;
  unsigned int* err = pkv::device_error_word(&st);
  if (st != PKV_OK) return st;

  Params p{};
  size_t off_o = 0, off_ml = 0;
  const size_t need = workspace_layout(batch, num_q_heads, head_dim, num_splits, info.sms, &off_o, &off_ml);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return PKV_EWORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PKV_EALIGN;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    p.counters = reinterpret_cast<int32_t*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + off_o);
    p.part_ml = reinterpret_cast<float*>(ws + off_ml);
  }
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
  p.scale_log2 = scale * 1.4426950408889634f;
  p.v_scale = 1.f;
  p.num_splits = num_splits;
  p.mod = mod;
  const int group = num_q_heads / num_kv_heads;
  if (dtype == PKV_BF16) {
    if (head_dim == 128) return dispatch_g<__nv_bfloat16, 128, kMod>(p, group, info.sms, stream);
    return dispatch_g<__nv_bfloat16, 64, kMod>(p, group, info.sms, stream);
  }
  if (head_dim == 128) return dispatch_g<float, 128, kMod>(p, group, info.sms, stream);
  return dispatch_g<float, 64, kMod>(p, group, info.sms, stream);
}

}  // namespace
