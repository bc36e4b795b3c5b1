// paged_decode_q4_kernel: decode, and chunks of at most 8 rows per KV head
// (kVar), over the 4-bit cache of q4.cuh.  The CTA plan, split and merge are
// decode_plan.cuh's.
//
// Bound: latency of the instructions between codes and products with two consumer
// warps per scheduler (issue slots 43 % busy, ALU pipe 39 %, tensor pipe 22 %, HBM 49 %
// over 32 sequences of 8192), then HBM (each token's K and V row once, 576 bytes each
// with 8 KV heads of 128).  256 sequences of 1k-8k tokens, 1.30 GB: 237 us, 5.5 TB/s;
// in copies of the kernel the stream alone takes 188 us, with only one of the two
// products 191-193.  At 4.5 bits an element the way from codes to matrix operands
// is what the kernel is built around:
//  * widen_q4 (q4.cuh): nine instructions for a word of eight codes.
//  * S^T = K Q^T: the 16 keys of a chunk in the M dimension and the R <= 8 rows
//    in N, so one m16n8k16 per 16 elements of head_dim wastes only the rows past
//    R.  A lane takes a whole quarter of its two keys' head rows (16 bytes each at
//    head_dim 128); q's fragments are laid out to match.
//  * O^T += V^T P^T: P^T's fragment is the transpose of S^T's, one movmatrix per
//    eight keys.  A lane takes 16 (head_dim 64: 8) consecutive elements of four keys:
//    one scale each.
//  * Both products see the softmax rows in the columns of their accumulators, so a
//    lane owns the state of rows 2c and 2c + 1 and rescaling needs no exchange.  A
//    row's reference moves when a score passes it by 15 (a vote per stage), to 7 below
//    the largest, so the usual stage takes no maximum across lanes.  The row sums are a
//    product of ones with the weights.
//  * f16 ends at 2^16, so a weight's exponent is the difference of the scaled score,
//    rounded to float32, and the reference, and that difference alone decides whether
//    the reference moves: no rounding of either, however large, lets a weight pass 2^15.
//    (A fused multiply and add would take the unrounded product.)
//  * Eight warps with four chunks of 16 keys each per stage: three chunks 244 us, two 258,
//    one 337 (four 235 in that measurement); 16 warps at 112 registers with two 250.
//  * Which token stands in which fragment row is free as long as K and V agree;
//    token_of spreads the rows over the banks.
// q enters as f16 after a power-of-two scaling of each row (as in the FP8 kernel);
// weights as f16 times 2^7, so that they count down to 2^-32 of the row's largest.
#pragma once

#include "decode_launch.cuh"
#include "decode_q4_args.cuh"
#include "q4.cuh"

namespace {

constexpr int kQ4Warps = 8;   // consumer warps (at most): one per (KV head, token phase)
constexpr int kQ4Stages = 6;  // at most
constexpr int kQ4Smem = 224 * 1024;
constexpr int kQ4Sub = 4;     // chunks of 16 keys per consumer warp and stage: their products overlap
constexpr int kQ4Chunk = 16 * kQ4Sub;
// Split points fall on multiples of this many tokens: parts of a few tokens cost more to
// merge than they save, large ones leave SMs idle (us at 1, 64, 128, 256: one sequence of
// 777 12.8, 12.9, 14.6, 16.8; 32 of 128-2048 24.9, 22.7, 24.9, 20.7; 4 of 32k-131k 85.2, 84.3,
// 83.1, 87.2).  A chunk has up to eight times the rows to merge (24 sequences of 1k-8k with 4
// drafted tokens: 54.9 at 64, 51.2 at 128).
constexpr int kQ4Align = 64;
constexpr int kQ4AlignChunk = 128;

// d (16x8 fp32) += a (16x16 f16, row) * b (16x8 f16, col)
__device__ __forceinline__ void mma_q4(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int kBytes>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[kBytes / 4]) {
  if constexpr (kBytes == 16)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
  else if constexpr (kBytes == 8)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}
template <int kBytes>  // 1 or 2
__device__ __forceinline__ uint32_t lds_short(uint32_t at) {
  uint32_t v;
  if constexpr (kBytes == 2)
    asm volatile("{\n\t.reg .u16 x;\n\tld.shared.u16 x, [%1];\n\tcvt.u32.u16 %0, x;\n\t}" : "=r"(v) : "r"(at));
  else
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
// Transposes an 8x8 matrix of 16-bit elements spread over the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// The token (of eight) that stands in fragment row i: rows i and i + 1, which one
// 16-byte load phase reads, differ in parity, and so do rows 0, 2, 4, 6 from one
// to the next, which V's loads take together (two rows of 8 heads of 128, 576
// bytes each, are 64 bytes apart modulo 128).
__device__ __forceinline__ int token_of(int i) { return i & 1 ? 4 + ((i >> 1) ^ 1) : i >> 1; }

constexpr int kChunkRows = 8;  // G * QL of the chunk instantiations

template <int G, int QL, int D, bool kVar>
__global__ void __launch_bounds__((kQ4Warps + 1) * 32, 1) paged_decode_q4_kernel(const Params p) {
  pkv::pdl_enter();
  {
    // warm L2 with small block tables while the plan reads the lengths
    const size_t lines = (static_cast<size_t>(p.batch) * p.max_blocks * 4 + 127) / 128;
    if (lines <= 512) {
      const char* tb = reinterpret_cast<const char*>(p.block_tables);
      for (size_t i = threadIdx.x; i < lines; i += blockDim.x)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(tb + i * 128) : "memory");
    }
  }
  using T = __nv_bfloat16;
  constexpr int R = G * QL;
  static_assert(R <= 8, "at most 8 rows per KV head");
  constexpr int NW = D / 32;   // code words of a lane's quarter of a key
  constexpr int NO = D / 16;   // m-tiles of O^T
  constexpr float kWeightLog2 = 7.0f;  // a row's largest weight when its reference is taken
  constexpr float kMost = 15.0f;       // and what one may grow to before it is taken again
  const int rows_per_seq = QL * p.hq;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x;
  const int warp = tid / 32;
  const int lane = tid % 32;
  const int nw = p.nw;
  const int hkv = p.hkv;
  const int row_bytes = pkv::q4_row_bytes(hkv, D);
  unsigned char* stage_base = smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(stage_base + p.stages * p.stage_bytes);
  uint64_t* empty = full + kQ4Stages;
  long long* sh = reinterpret_cast<long long*>(empty + kQ4Stages);
  int* sh_flag = reinterpret_cast<int*>(sh + 64);
  float* merge = reinterpret_cast<float*>(sh_flag + 32);  // records of the phases past the first
  volatile int* abort_flag = sh_flag + 1;
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < p.stages; ++s) {
      pkv::mbar_init(&full[s], 1);
      pkv::mbar_init(&empty[s], nw);
    }
    pkv::fence_mbar_init();
  }
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (covered_len<true, kVar>(p, b) != 0) continue;
    int first = b * rows_per_seq, count = rows_per_seq;
    if constexpr (kVar) {
      if (seq_len<kVar>(p, b) == 0) continue;  // no rows, or skipped
      first = __ldg(p.cu_q + b) * p.hq;
      count = (__ldg(p.cu_q + b + 1) - __ldg(p.cu_q + b)) * p.hq;
    }
    T* o = static_cast<T*>(p.out) + static_cast<size_t>(first) * D;
    for (int i = tid; i < count * D; i += blockDim.x) o[i] = static_cast<T>(0.0f);
  }
  Plan plan;
  if (p.num_splits > 0) {
    plan_fixed<true>(p, plan);
    __syncthreads();
  } else {
    plan_auto<true, kVar>(p, plan, sh);
  }

  if (warp == nw) {
    // ------------------------------------------------------------ producer
    // A stage's tokens are contiguous runs of rows, one per block: a copy of K and
    // one of V per run, a run per lane.
    const uint64_t policy = pkv::l2_evict_first_policy();
    int s = 0;
    uint32_t parity = 1;  // (a ring's first pass finds every stage free)
    for_each_segment<true, kVar>(p, plan, [&](const Segment& seg) -> bool {
      const int32_t* table = p.block_tables + static_cast<size_t>(seg.b) * p.max_blocks;
      for (int t = seg.t0; t < seg.t1; t += p.t_stage) {
        const int end = min(t + p.t_stage, seg.t1);
        const int last = (end - 1) / p.block_size;
        const int first = t / p.block_size + lane;
        int phys = first <= last ? __ldg(table + first) : 0;
        if (lane == 0) wait_or_abort(&empty[s], parity, abort_flag, p.err);
        __syncwarp();
        for (int blk = first; blk <= last; blk += 32) {
          if (blk != first) phys = __ldg(table + blk);
          if (phys < 0 || phys >= p.num_blocks) {
            pkv::raise_error(p.err, PKV_DERR_BLOCK_RANGE);
            continue;
          }
          const int a = max(t, blk * p.block_size);
          const uint32_t bytes = static_cast<uint32_t>(min(end - a, (blk + 1) * p.block_size - a)) * row_bytes;
          const size_t src =
              (static_cast<size_t>(phys) * p.block_size + (a - blk * p.block_size)) * static_cast<size_t>(row_bytes);
          unsigned char* dst = stage_base + s * p.stage_bytes + (a - t) * row_bytes;
          pkv::mbar_expect_tx(&full[s], 2 * bytes);
          pkv::bulk_g2s(dst, p.k_cache + src, bytes, &full[s], policy);
          pkv::bulk_g2s(dst + p.stage_bytes / 2, p.v_cache + src, bytes, &full[s], policy);
        }
        __syncwarp();
        if (lane == 0) pkv::mbar_arrive(&full[s]);
        if (++s == p.stages) {
          s = 0;
          parity ^= 1u;
        }
      }
      return true;
    });
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = warp % hkv;
  const int phase = warp / hkv;
  const int r0 = lane >> 2;  // fragment rows r0 and r0 + 8 (keys of S^T, elements of O^T); column r0 of B operands
  const int c = lane & 3;
  const int nthreads_c = nw * 32;
  const int tw0 = phase * kQ4Chunk;  // this warp's keys of a stage
  // offsets in a stage of what this lane reads: two keys' quarter and scales, four V rows' elements and scales
  const int scales = pkv::q4_scale_offset(hkv, D) + g * (D / 16);
  const int k_at = (tw0 + token_of(r0)) * row_bytes;
  const int k_codes = k_at + g * (D / 2) + c * (D / 8);
  const int k_scales = k_at + scales + c * (D / 64);
  const int va = token_of(2 * c), vb = token_of(2 * c + 1);
  const int v_a = (tw0 + va) * row_bytes, v_b = (tw0 + vb) * row_bytes;
  const int v_codes = g * (D / 2) + r0 * (D / 16);
  const int v_scales = scales + (D == 128 ? r0 : r0 >> 1);
  const int half = 8 * row_bytes;  // from fragment rows r0 to r0 + 8
  const uint32_t ring = pkv::smem_u32(stage_base);
  const uint32_t stage_bytes = static_cast<uint32_t>(p.stage_bytes);
  int stage = 0;
  uint32_t at = ring;  // the stage's K rows, its V rows half a stage further
  uint32_t parity = 0;

  for_each_segment<true, kVar>(p, plan, [&](const Segment& seg) -> bool {
    // Q as the B operand: column r0, and for word w of this lane's quarter the pairs (0, 4), (1, 5), (2, 6), (3, 7)
    uint32_t qf[NW][4];
    float mul[2];  // of rows 2c and 2c + 1: the power that scaled q comes off with the scale (and K's unit)
    {
      const bool row_here = kVar ? r0 / G < seg.nq && r0 < R : r0 < R;
      const size_t row = kVar ? static_cast<size_t>(seg.q0) + r0 / G : static_cast<size_t>(seg.b) * QL + r0 / G;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (row * p.hq + g * G + r0 % G) * D +
                                                        c * (D / 4));
      float f[NW][8];
      float amax = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const uint4 x = row_here ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
        Chunk<T>::unpack(x, f[w]);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[w][i]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int ex = amax > 0.f ? min(max(14 - ilogbf(amax), -113), 126) : 0;
      const float up = copysignf(pkv::power_of_two(ex), p.scale_log2);  // (the scale's sign goes with q)
      const float down = pkv::row_scale(fabsf(p.scale_log2), p.scale_exp - ex);
      mul[0] = __shfl_sync(0xffffffffu, down, 8 * c);
      mul[1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[w][i] = pkv::pack_f16x2(f[w][i] * up, f[w][i + 4] * up);
    }
    int lim[2] = {seg.ctx - 1, seg.ctx - 1};  // the last key that rows 2c and 2c + 1 see
    if constexpr (kVar) {
      if (p.causal)
#pragma unroll
        for (int i = 0; i < 2; ++i) lim[i] = seg.ctx - seg.nq + (2 * c + i) / G;
    }
    float o[NO][4];
#pragma unroll
    for (int j = 0; j < NO; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    // the rows' references, what an exponent starts from (kNoScore, below every score: none yet)
    constexpr float kNoScore = -FLT_MAX;
    float base[2] = {kNoScore, kNoScore};
    float l[4] = {0.f, 0.f, 0.f, 0.f};  // of rows 2c and 2c + 1, twice: a product of ones with the weights

    for (int t = seg.t0; t < seg.t1; t += p.t_stage) {
      if (!pkv::mbar_try_wait(&full[stage], parity)) wait_or_abort(&full[stage], parity, abort_flag, p.err);
      const int nv = min(seg.t1 - t - tw0, kQ4Chunk);  // keys of this warp in the stage
      if (nv > 0) {
        const uint32_t kc = at + k_codes, ks = at + k_scales;
        const uint32_t vs = at + stage_bytes / 2;
        float x[kQ4Sub][4];
#pragma unroll
        for (int u = 0; u < kQ4Sub; ++u) {
          uint32_t wx[NW], wy[NW];  // keys r0 and r0 + 8
          lds_words<D / 8>(kc + 2 * u * half, wx);
          lds_words<D / 8>(kc + (2 * u + 1) * half, wy);
          const uint32_t sx = lds_short<D / 64>(ks + 2 * u * half), sy = lds_short<D / 64>(ks + (2 * u + 1) * half);
          const uint32_t hx = pkv::e4m3x2_to_f16x2(sx), hy = pkv::e4m3x2_to_f16x2(sy);  // the quarter's groups
#pragma unroll
          for (int e = 0; e < 4; ++e) x[u][e] = 0.f;
#pragma unroll
          for (int grp = 0; grp < NW / 2; ++grp) {
            const pkv::Q4Scale kx(pkv::prmt(hx, 0, grp ? 0x3232u : 0x1010u)), ky(pkv::prmt(hy, 0, grp ? 0x3232u : 0x1010u));
#pragma unroll
            for (int w = 2 * grp; w < 2 * grp + 2; ++w) {
              uint32_t fx[4], fy[4];
              pkv::widen_q4(wx[w], kx, fx);
              pkv::widen_q4(wy[w], ky, fy);
              mma_q4(x[u], fx[0], fy[0], fx[1], fy[1], qf[w][0], qf[w][1]);
              mma_q4(x[u], fx[2], fy[2], fx[3], fy[3], qf[w][2], qf[w][3]);
            }
          }
        }
        // raw scores of keys r0 (e = 0, 1) and r0 + 8 (2, 3) of each chunk for rows 2c and 2c + 1, then scaled
        float top[2] = {-INFINITY, -INFINITY};
        const bool partial = nv < kQ4Chunk;
        if (partial || (kVar && t + tw0 + kQ4Chunk > seg.ctx - seg.nq)) {
#pragma unroll
          for (int u = 0; u < kQ4Sub; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = t + tw0 + 16 * u + token_of(r0) + (e >= 2 ? 8 : 0);
              if (key >= seg.t1 || key > lim[e & 1]) x[u][e] = -INFINITY;
            }
        }
        const uint64_t muls = pkv::pair(mul[0], mul[1]);
#pragma unroll
        for (int u = 0; u < kQ4Sub; ++u)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            pkv::split(pkv::mul2(pkv::pair(x[u][e], x[u][e + 1]), muls), x[u][e], x[u][e + 1]);
            top[0] = fmaxf(top[0], x[u][e]);
            top[1] = fmaxf(top[1], x[u][e + 1]);
          }
        if (__any_sync(0xffffffffu, top[0] - base[0] > kMost || top[1] - base[1] > kMost)) {
          // (a row moves by its own scores only)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mx = top[i];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            if (mx - base[i] > kMost) {
              const float next = mx - kWeightLog2;
              const float corr = pkv::ex2(base[i] - next);  // 0 while there is no score
              base[i] = next;
              l[i] *= corr;
              l[2 + i] *= corr;
#pragma unroll
              for (int j = 0; j < NO; ++j) {
                o[j][i] *= corr;
                o[j][2 + i] *= corr;
              }
            }
          }
        }
        uint32_t pf[kQ4Sub][2];  // weights of keys r0 and r0 + 8, then of this lane's V rows
        const uint64_t from = pkv::pair(-base[0], -base[1]);
#pragma unroll
        for (int u = 0; u < kQ4Sub; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float a, b;
            pkv::split(pkv::add2(pkv::pair(x[u][2 * i], x[u][2 * i + 1]), from), a, b);
            pf[u][i] = movmatrix(pkv::pack_f16x2(pkv::ex2(a), pkv::ex2(b)));
          }
#pragma unroll
        for (int u = 0; u < kQ4Sub; ++u) {
          constexpr uint32_t kOnes = 0x3c003c00u;
          mma_q4(l, kOnes, kOnes, kOnes, kOnes, pf[u][0], pf[u][1]);
          const uint32_t va_at = vs + v_a, vb_at = vs + v_b;
          const int lo = 2 * u * half, hi = lo + half;
          uint32_t s_ab = lds_short<1>(va_at + v_scales + lo) + lds_short<1>(vb_at + v_scales + lo) * 256u;
          uint32_t s_cd = lds_short<1>(va_at + v_scales + hi) + lds_short<1>(vb_at + v_scales + hi) * 256u;
          if (partial) {  // rows past the last key hold anything: scale 0 makes their values 0
            const int n = nv - 16 * u;
            s_ab &= (va < n ? 0x00ffu : 0u) | (vb < n ? 0xff00u : 0u);
            s_cd &= (va + 8 < n ? 0x00ffu : 0u) | (vb + 8 < n ? 0xff00u : 0u);
          }
          const pkv::Q4Scale kab(pkv::e4m3x2_to_f16x2(s_ab)), kcd(pkv::e4m3x2_to_f16x2(s_cd));
          uint32_t wv[4][NW / 2];
          lds_words<D / 16>(va_at + v_codes + lo, wv[0]);
          lds_words<D / 16>(vb_at + v_codes + lo, wv[1]);
          lds_words<D / 16>(va_at + v_codes + hi, wv[2]);
          lds_words<D / 16>(vb_at + v_codes + hi, wv[3]);
#pragma unroll
          for (int w = 0; w < NW / 2; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // four elements of keys (2c, 2c + 1) and of (2c + 8, 2c + 9), a pair of keys per word
              uint32_t fab[4], fcd[4];
              pkv::widen_q4(pkv::prmt(wv[0][w], wv[1][w], h ? 0x7632u : 0x5410u), kab, fab);
              pkv::widen_q4(pkv::prmt(wv[2][w], wv[3][w], h ? 0x7632u : 0x5410u), kcd, fcd);
              const int tm = 4 * w + 2 * h;
              mma_q4(o[tm], fab[0], fab[1], fcd[0], fcd[1], pf[u][0], pf[u][1]);
              mma_q4(o[tm + 1], fab[2], fab[3], fcd[2], fcd[3], pf[u][0], pf[u][1]);
            }
        }
      }
      __syncwarp();
      if (lane == 0) pkv::mbar_arrive(&empty[stage]);
      at += stage_bytes;
      if (++stage == p.stages) {
        stage = 0;
        at = ring;
        parity ^= 1u;
      }
    }
    float m[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i] = base[i] == kNoScore ? -INFINITY : base[i];  // (sums are relative to it)
    // accumulator (tm, i) is element d0 + 2 tm of row 2c + i, (tm, 2 + i) the next one
    const int d0 = r0 * (D / 8);
    if (p.wph > 1) {
      // merge the warps that share KV head g
      constexpr int rec = D + 2;
      float* mine = merge + static_cast<size_t>(warp - p.hkv) * R * rec;
      if (phase > 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 2 * c + i;
          if (row >= R) continue;
#pragma unroll
          for (int tm = 0; tm < NO; ++tm)
            *reinterpret_cast<float2*>(mine + row * rec + d0 + 2 * tm) = make_float2(o[tm][i], o[tm][2 + i]);
          if (r0 == 0) *reinterpret_cast<float2*>(mine + row * rec + D) = make_float2(m[i], l[i]);
        }
      }
      pkv::named_barrier_sync(1, nthreads_c);
      if (phase == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 2 * c + i;
          if (row >= R) continue;
          float mm = m[i];
          for (int ph = 1; ph < p.wph; ++ph)
            mm = fmaxf(mm, merge[(static_cast<size_t>((ph - 1) * p.hkv + g) * R + row) * rec + D]);
          const float w0 = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mm);
          float ll = l[i] * w0;
#pragma unroll
          for (int tm = 0; tm < NO; ++tm) {
            o[tm][i] *= w0;
            o[tm][2 + i] *= w0;
          }
          for (int ph = 1; ph < p.wph; ++ph) {
            const float* src = merge + (static_cast<size_t>((ph - 1) * p.hkv + g) * R + row) * rec;
            const float w = src[D] == -INFINITY ? 0.f : exp2f(src[D] - mm);
            ll += w * src[D + 1];
#pragma unroll
            for (int tm = 0; tm < NO; ++tm) {
              const float2 v = *reinterpret_cast<const float2*>(src + d0 + 2 * tm);
              o[tm][i] = fmaf(w, v.x, o[tm][i]);
              o[tm][2 + i] = fmaf(w, v.y, o[tm][2 + i]);
            }
          }
          m[i] = mm;
          l[i] = ll;
        }
      }
      pkv::named_barrier_sync(1, nthreads_c);
    }
    // the result (whole sequence) or this part's state; V's scale comes off here (the weights' 2^7 cancels against l)
    if (phase == 0) {
      const float vscale = p.v_scale * pkv::kQ4Unit;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 2 * c + i;
        if (row >= R || (kVar && row / G >= seg.nq)) continue;
        const int head = (row / G) * p.hq + g * G + row % G;
        if (seg.nparts == 1) {
          const float inv = l[i] == 0.f ? 0.f : vscale / l[i];  // kVar: a row may see nothing
          T* orow = static_cast<T*>(p.out) + ((kVar ? static_cast<size_t>(seg.q0) * p.hq
                                                    : static_cast<size_t>(seg.b) * rows_per_seq) + head) * D + d0;
          uint32_t w[NO];
#pragma unroll
          for (int tm = 0; tm < NO; ++tm) w[tm] = pkv::pack_bf16x2(o[tm][i] * inv, o[tm][2 + i] * inv);
#pragma unroll
          for (int u = 0; u < NO / 4; ++u)
            reinterpret_cast<uint4*>(orow)[u] = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
        } else {
          float* po = p.part_o + (static_cast<size_t>(seg.slot) * rows_per_seq + head) * D + d0;
#pragma unroll
          for (int u = 0; u < NO / 2; ++u)
            reinterpret_cast<float4*>(po)[u] = make_float4(o[2 * u][i] * vscale, o[2 * u][2 + i] * vscale,
                                                           o[2 * u + 1][i] * vscale, o[2 * u + 1][2 + i] * vscale);
          if (r0 == 0)
            *reinterpret_cast<float2*>(p.part_ml + (static_cast<size_t>(seg.slot) * rows_per_seq + head) * 2) =
                make_float2(m[i], l[i]);
        }
      }
    }
    if (seg.nparts > 1) combine_if_last<T, D, true, kVar>(p, seg, rows_per_seq, sh_flag, nthreads_c);
    return true;
  });
}

// ------------------------------------------------------------------ host side

template <int G, int QL, int D, bool kVar>
int launch_q4(Params& p, int sms, cudaStream_t stream) {
  constexpr int R = G * QL;
  const int row = pkv::q4_row_bytes(p.hkv, D);
  p.wph = kQ4Warps / p.hkv;
  p.nw = p.hkv * p.wph;
  p.t_stage = kQ4Chunk * p.wph;
  p.stage_bytes = static_cast<size_t>(p.t_stage) * row * 2;
  p.align = kVar ? kQ4AlignChunk : kQ4Align;
  const size_t misc = 2 * kQ4Stages * sizeof(uint64_t) + 64 * sizeof(long long) + 32 * sizeof(int) +
                      static_cast<size_t>(p.nw - p.hkv) * R * (D + 2) * sizeof(float);
  p.stages = std::min<int>(kQ4Stages, static_cast<int>((kQ4Smem - misc) / p.stage_bytes));
  if (p.stages < 2) return PKV_EUNSUPPORTED;
  auto kernel = paged_decode_q4_kernel<G, QL, D, kVar>;
  static std::atomic<uint64_t> smem_allowed{0};  // the limit for every number of KV heads
  if (pkv::allow_smem(kernel, kQ4Smem, smem_allowed) != cudaSuccess) return PKV_ECUDA;
  const unsigned grid = p.num_splits > 0 ? static_cast<unsigned>(static_cast<long long>(p.batch) * p.num_splits)
                                         : static_cast<unsigned>(sms * kAutoCtasPerSm);
  if (grid == 0) return PKV_OK;
  return pkv::launch_pdl(kernel, dim3(grid), dim3((p.nw + 1) * 32), p.stages * p.stage_bytes + misc, stream, p) ==
                 cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

template <int D, bool kVar>
int dispatch_q4(Params& p, int group, int sms, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_q4<1, kVar ? kChunkRows : 1, D, kVar>(p, sms, stream);
    case 2: return launch_q4<2, kVar ? kChunkRows / 2 : 1, D, kVar>(p, sms, stream);
    case 4: return launch_q4<4, kVar ? kChunkRows / 4 : 1, D, kVar>(p, sms, stream);
    default: return launch_q4<8, 1, D, kVar>(p, sms, stream);
  }
}

template <int D>
int run_q4(const pkv::Q4Decode& a, cudaStream_t stream) {
  const bool chunk = a.cu_q != nullptr;
  pkv::DeviceInfo info;
  if (pkv::device_info(&info) != PKV_OK) return PKV_ECUDA;
  Params p{};
  size_t off_o = 0, off_ml = 0;
  const size_t need = workspace_layout(a.batch, chunk ? kChunkRows * a.hkv : a.hq, D, a.num_splits, info.sms, &off_o, &off_ml);
  if (need > 0) {
    if (!a.workspace || a.workspace_bytes < need) return PKV_EWORKSPACE;
    if ((reinterpret_cast<uintptr_t>(a.workspace) & 255u) != 0) return PKV_EALIGN;
    unsigned char* ws = static_cast<unsigned char*>(a.workspace);
    p.counters = reinterpret_cast<int32_t*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + off_o);
    p.part_ml = reinterpret_cast<float*>(ws + off_ml);
  }
  p.out = a.out;
  p.q = a.q;
  p.k_cache = static_cast<const unsigned char*>(a.k_cache);
  p.v_cache = static_cast<const unsigned char*>(a.v_cache);
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.err = a.err;
  p.max_blocks = a.max_blocks;
  p.batch = a.batch;
  p.hq = a.hq;
  p.ql = 1;
  p.hkv = a.hkv;
  p.block_size = a.block_size;
  p.num_blocks = a.num_blocks;
  p.scale_log2 = pkv::split_scale(a.scale, a.k_scale * pkv::kQ4Unit, &p.scale_exp);
  p.v_scale = a.v_scale;
  p.num_splits = a.num_splits;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.total_q = a.total_q;
  p.max_seqlen_q = a.max_seqlen_q;
  p.causal = a.causal;
  const int group = a.hq / a.hkv;
  return chunk ? dispatch_q4<D, true>(p, group, info.sms, stream) : dispatch_q4<D, false>(p, group, info.sms, stream);
}

}  // namespace
