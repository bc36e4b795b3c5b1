// paged_varlen_prefill_attn on the 5th-generation tensor cores (tcgen05).
//
// What is computed is the same as the mma.sync kernel in prefill.cu
// ("3.6 ModelRunner, CUDA Graph, and benchmarks", section 2, prepare_prefill):
// query row r of sequence i sits at absolute position c + r (c = nk - nq
// history tokens) and, causally, attends keys 0..c + r, read through the
// block table (or from the packed k/v rows when there is no history).
//
// How: one CTA per SM owns a pair of query tiles of one (sequence, KV head):
// tile A and the tile after it, B.  A tile's 128 rows are (token, query head
// of the KV group) pairs, token-major, so one TMA box of q covers them and
// every K/V tile serves all G heads of both query tiles.
//   warp 0     TMA producer (one thread): Q of both tiles once, then K and V
//              tiles of 128 keys into 2-stage rings (128-byte swizzled, one
//              box per 64-wide d slab; paged tiles are gathered block piece by
//              block piece).  Then the whole warp zeroes the V rows past the
//              last key in the last tile before the MMA thread may use it.
//   warp 1     MMA issuer: the whole warp runs the loop, one elected lane
//              issues each group of MMAs from one asm block, so the issuing
//              work stays warp-uniform and short (the warp shares its SMSP with
//              four busy softmax warps).  Per key tile j the tensor pipe runs
//                 P_A(j) V(j),  Q_A K(j+1)^T,  P_B(j) V(j),  Q_B K(j+1)^T
//              (each a group of eight M=128, N=128 MMAs), so each tile's
//              softmax has the other tile's two groups to hide behind.  S and
//              O of both tiles sit in TMEM (4 x 128 columns); P is written
//              over S in bf16 and read from TMEM as the A operand of P V.
//   warps 2-9  softmax of tile A, two threads per TMEM lane (= query row),
//              one per half of the key tile: scale, mask, row max (the two
//              warps on the same 32 rows exchange theirs through shared memory
//              at a 64-thread named barrier), exp2, bf16 P; O is
//              rescaled in TMEM only when the row max grows by more than 2^8;
//              final normalisation and store (each half 64 of the 128 columns).
//   warps 10-17  the same for tile B.
// Why this shape (measured on GB300): one issuing thread needs about 45
// cycles per tcgen05.mma whatever its N, and each barrier wait between MMA
// groups idles the pipe for ~100 cycles; four groups of N = 128 per key tile
// keep it busy ~83 % of the time even so, where 32- or 64-key tiles per
// query tile reached a fifth to a half.  The pair shares every K/V tile,
// halving the load bytes per flop.
// Every wait is bounded; on a timeout the CTA records an error, skips the
// remaining waits and still frees its TMEM.
//
// Further forms of the kernel share this file (Form below; each is instantiated
// in a file of its own):
//   kMod   score modifiers.  The key tiles of a pair start at its rows' least
//          first key and end at its largest visible key (a prefix may reach past
//          the causal end).  Masks alone (kMasked), with a cap (kCapped), with a
//          distance bias (kBiased) or both are separate instantiations: a thread
//          holds its 64 scores in registers at a cap of 96, and one kernel that
//          branched on the modifiers at run time spilled (a batch of 16 chunks,
//          56 GFLOP, no modifier given: 70.7 us against the plain kernel's 62.6).
//   kFp8   an E4M3 cache: a tile's codes arrive in part of its K or V stage, and
//          two more warps widen them to f16 in place, a quarter of the tile (32
//          keys) at a time through registers.  (A ring of its own for the codes
//          fitted three half tiles; the loads in flight bounded it: a batch of 16
//          chunks, 56 GFLOP, 79 us.)
//   kInt4  a 4-bit cache: three warps (the producer's, which has only Q to load, is
//          one) widen rows to f16, a lane per row and a quarter of a tile (32 keys)
//          at a time.  A warp copies its quarters' codes and scales into a ring of
//          its own, three quarters ahead (rows and scales need not suit a tensor
//          copy).  The four pairs of a code word are stored as they come out,
//          elements (0, 4), (1, 5), (2, 6), (3, 7): the rewritten Q has the same
//          order, the epilogue undoes it for V.
//          A batch of 16 chunks, 56 GFLOP, 78 us (the E4M3 form 74); when it took 86, in
//          copies of the kernel 76 without the loads, 72 without the widening, 66
//          without both.  (Rows copied by their own lanes, 16 bytes at a time, 91.)
#pragma once

#include <algorithm>
#include <cfloat>

#include "prefill_args.cuh"
#include "q4.cuh"
#include "tcgen05.cuh"

namespace {

using namespace pkv;

constexpr int kBM = 128;   // rows per query tile
constexpr int kBN = 128;   // keys per tile
constexpr int kStages = 2; // K ring and V ring depth
constexpr int kSoftmaxWarps = 8;  // per query tile: two threads per row, one per half of the key tile
constexpr int kWidenWarps = 2;    // kFp8, kInt4: warps that widen codes to f16 (kInt4: and warp 0)
enum Form { kPlain, kMasked, kCapped, kBiased, kCappedBiased, kE4m3, kInt4 };
__host__ __device__ constexpr bool quantized(Form f) { return f == kE4m3 || f == kInt4; }
__host__ __device__ constexpr int threads(Form f) { return 32 * (2 + 2 * kSoftmaxWarps + (quantized(f) ? kWidenWarps : 0)); }
constexpr int kQuarter = 32;  // kFp8, kInt4: keys widened at a time
constexpr int kInt4Depth = 4;  // kInt4: quarters in a widening warp's ring
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;    // S_A at 0, S_B at 128
constexpr uint32_t kColO = 256;  // O_A at 256, O_B at 384
constexpr uint32_t kSlabQ = kBM * 128;
constexpr uint32_t kSlabKV = kBN * 128;
constexpr uint32_t kRedBytes = 2 * 2 * 2 * kBM * 4;  // row maxima / sums exchanged by the halves: [tile parity][query tile][half][row]

// Sizes for head dimension D (64 or 128): a row of D bf16 is D / 64 slabs of
// 128 bytes (one 128-byte swizzle atom each), and each slab of a tile is a
// TMA box of its own.
template <int D>
struct Geo {
  static_assert(D == 64 || D == 128, "head_dim 64 or 128");
  static constexpr int kSlabs = D / 64;
  static constexpr uint32_t kTileQ = kSlabs * kSlabQ;
  static constexpr uint32_t kTileKV = kSlabs * kSlabKV;
  static constexpr uint32_t kRedOffset = 2 * kTileQ + 2 * kStages * kTileKV;
  static constexpr uint32_t kBarOffset = kRedOffset + kRedBytes;
  static constexpr uint32_t kSmemBytes = kBarOffset + 256 + 1024;  // barriers + 1 KB for alignment
  // kInt4: the rings of codes, then of scales, follow the barriers
  static constexpr uint32_t kInt4Codes = kQuarter * D / 2;
  static constexpr uint32_t kInt4Slot = kInt4Codes + kQuarter * D / 16;
  static constexpr uint32_t kInt4Offset = kBarOffset + 256;
  static constexpr uint32_t kInt4Bytes = (kWidenWarps + 1) * kInt4Depth * kInt4Slot;
  // one CTA per SM even when two would fit (each holds all 512 TMEM columns)
  static constexpr uint32_t launch_smem(Form f) {
    return std::max<uint32_t>(kSmemBytes + (f == kInt4 ? kInt4Bytes : 0), 120 * 1024);
  }
  static constexpr size_t kRecordBytes = static_cast<size_t>(kBM) * D * 4 + static_cast<size_t>(kBM) * 8;
};
static_assert(Geo<128>::launch_smem(kInt4) <= 227 * 1024, "shared memory plan exceeds an SM");
constexpr float kRescaleLog2 = 8.0f;
// kFp8, kInt4: weights enter P V as f16, whose subnormals end at 2^-24, so they are taken 2^7 times
// as large (with the lazy rescale at most 2^15): a weight then counts down to 2^-32 of the
// row's largest.  Without the factor 131072 keys 17.4 below a dominant one, 0.36 % of the
// mass, came out as nothing.
constexpr float kF16WeightLog2 = 7.0f;

// Key-range split of long work items, used only when the pairs do not fill
// the GPU (small batches with long histories) and a workspace is given.  With
// P parts chosen on the host, a pair with more than kSplitMinTiles key tiles
// runs as up to P CTAs over consecutive ranges of its key tiles.  For each of
// its two query tiles, every part but the last to finish publishes its
// unnormalised O and its row maxima and sums (one record per part); the last
// merges the records and its own TMEM result by the log-sum-exp rule, in part
// order, and stores the output.
constexpr int kSplitMinTiles = 8;
constexpr int kMaxParts = 8;
constexpr uint64_t kSplitWaitNs = 1000000000ull;  // bound on the last part's wait for the records

// Per query tile X (A = 0, B = 1): S_FULL + X completes when S_X holds the
// scores of the next key tile (and so every P_X V issued before it has
// completed too), P_FULL + X when its softmax warps have written P over it.
// O_FINAL + X completes once, after the last P_X V: tile X's epilogue waits on
// it (A's can start while B still runs).  K and V stages are released
// separately, a K stage once both Q K^T products have read it, a V stage once
// both P V products have.  V_TAIL: the last V tile, once its rows past the
// last key are zeroed (only when that tile is partial).
enum Bar {
  Q_FULL = 0,
  K_FULL = 1,
  V_FULL = K_FULL + kStages,
  K_EMPTY = V_FULL + kStages,
  V_EMPTY = K_EMPTY + kStages,
  S_FULL = V_EMPTY + kStages,
  P_FULL = S_FULL + 2,
  O_FINAL = P_FULL + 2,  // per query tile
  V_TAIL = O_FINAL + 2,
  V_HEAD,  // kMod: the first V tile, once its rows before the first visible key are zeroed
  Q_READY,  // kFp8, kInt4, per query tile: Q rewritten as scaled f16
  RAW_FULL = Q_READY + 2,  // kFp8, per K stage, then per V stage: the codes have arrived
  NUM_BARS = RAW_FULL + 2 * kStages
};
static_assert(NUM_BARS * 8 + 16 <= 256, "barrier area too small");

// c log2e tanh(k s) of a raw score s as s P(s^2), k = raw_to_x: P of degree 2
// for |k s| <= 0.4 and of degree 4 for |k s| <= 1.  The coefficients of tanh(x) / x
// minimise its largest relative error (a reweighted least-squares fit), 6.2e-6
// and 6.9e-6: a score of 20 is off by 1.2e-4 or less, which changes a weight by a
// thirtieth of its bf16 rounding.  c log2e and the powers of k are folded in; a
// tier whose coefficients leave fp32's normal range is not used.
struct TanhPoly {
  float near[3];
  float wide[5];
  float near_limit;  // raw scores up to here take `near`, up to wide_limit `wide` (-infinity: tier not used)
  float wide_limit;
};

inline TanhPoly make_tanh_poly(float cap_log2, float k) {
  constexpr double near[3] = {0.9999937531147292, -0.3326257940886756, 0.12127786248978804};
  constexpr double wide[5] = {0.9999930893432413, -0.3329806519023404, 0.13036811004581145, -0.04481755092515754,
                              0.009036422447889145};
  TanhPoly p{};
  bool near_ok = true, wide_ok = true;
  double power = static_cast<double>(cap_log2) * k;
  for (int i = 0; i < 5; ++i) {
    if (i < 3) {
      p.near[i] = static_cast<float>(near[i] * power);
      near_ok = near_ok && std::isnormal(p.near[i]);
    }
    p.wide[i] = static_cast<float>(wide[i] * power);
    wide_ok = wide_ok && std::isnormal(p.wide[i]);
    power *= static_cast<double>(k) * k;
  }
  // (scores whose squares overflow are beyond both: 1 / k < 2^60)
  const bool square_ok = k > 0x1p-60f;
  p.near_limit = near_ok && square_ok ? 0.4f / k : -INFINITY;
  p.wide_limit = wide_ok && square_ok ? 1.0f / k : -INFINITY;
  // an unused tier still sees tiles in which every key is hidden: any positive
  // polynomial keeps -infinity
  if (!near_ok) std::fill_n(p.near, 3, 1.f);
  if (!wide_ok) std::fill_n(p.wide, 5, 1.f);
  return p;
}

struct TcParams {
  __nv_bfloat16* out;
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* block_tables;
  unsigned int* err;
  int total_q;
  int total_k;
  int max_seqlen_q;
  int max_blocks;
  int hq;
  int hkv;
  int block_size;
  int num_blocks;
  float scale_log2;  // scale * log2(e); kFp8, kInt4: times 2^scale_exp that, times the K scale
  int causal;
  int paged;
  int piece_rows;  // rows per K/V TMA box (paged: min(block_size, kBN))
  int q_tiles;     // query tiles per sequence, rounded up to a whole number of pairs
  int parts_max;   // P: the most parts a long pair runs as (1: no split)
  int* tickets;    // [sequences x KV heads x q_tiles]: finish order of a split tile's parts, reset by the last
  int* ready;      // [same]: records published so far, reset by the last
  unsigned char* records;  // [same][P][record bytes]: O (D / 4 chunks of 4 fp32 columns x kBM rows), then m[kBM], l[kBM]
  ScoreMod mod;            // kMod
  TanhPoly tanh_poly;      // kMod with a cap
  float bias_mul;          // slopes to the units of bias_scores
  const unsigned char* k_codes;  // kInt4: the pools; kFp8: for block sizes whose pieces are single rows
  const unsigned char* v_codes;
  float v_scale;
  uint32_t block_mul;  // kInt4: key / block_size = key * block_mul >> block_shift
  int block_shift;
  int scale_exp;
};

}  // namespace

namespace {

struct Waiter {
  volatile int* abort_flag;
  unsigned int* err;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) const {
    // one try_wait first: no shared-memory read of the abort flag on the fast path
    if (mbar_try_wait(bar, parity)) return;
    slow(bar, parity);
  }
  // For phases that have usually completed already (loads issued long
  // before): a test_wait returns at once.
  __device__ __forceinline__ void ready(uint64_t* bar, uint32_t parity) const {
    if (mbar_test_wait(bar, parity)) return;
    if (mbar_try_wait(bar, parity)) return;
    slow(bar, parity);
  }
  __device__ __noinline__ void slow(uint64_t* bar, uint32_t parity) const {
    if (*abort_flag) return;
    if (!mbar_wait(bar, parity)) {
      *abort_flag = 1;
      raise_error(err, PKV_DERR_WAIT_TIMEOUT);
    }
  }
};

// exp2(scale * s - m) for two scores (fma on the f32x2 pair, ex2.approx per
// element), rounded to bf16 and packed low = first; the two rounded values are
// added to the row-sum lanes acc (widened exactly: fma by 1 in fp32).
__device__ __forceinline__ uint32_t exp2_pair_bf16(uint32_t s0, uint32_t s1, float scale, float neg_m,
                                                   uint64_t& acc) {
  uint32_t out;
  asm("{\n\t.reg .b64 x, c, m;\n\t.reg .f32 a, b, sa, sb;\n\t.reg .b16 pa, pb, one;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 c, {%4, %4};\n\t"
      "mov.b64 m, {%5, %5};\n\t"
      "fma.rn.f32x2 x, x, c, m;\n\t"
      "mov.b64 {a, b}, x;\n\t"
      "ex2.approx.ftz.f32 a, a;\n\t"
      "ex2.approx.ftz.f32 b, b;\n\t"
      "cvt.rn.bf16x2.f32 %0, b, a;\n\t"
      "mov.b32 {pa, pb}, %0;\n\t"
      "mov.b16 one, 0x3f80;\n\t"
      "mov.b64 {sa, sb}, %1;\n\t"
      "fma.rn.f32.bf16 sa, pa, one, sa;\n\t"
      "fma.rn.f32.bf16 sb, pb, one, sb;\n\t"
      "mov.b64 %1, {sa, sb};\n\t}"
      : "=r"(out), "+l"(acc)
      : "r"(s0), "r"(s1), "f"(scale), "f"(neg_m));
  return out;
}

// The same with f16 weights (kFp8, kInt4), which reach 2^15 (kF16WeightLog2 and the lazy rescale).
__device__ __forceinline__ uint32_t exp2_pair_f16(uint32_t s0, uint32_t s1, float scale, float neg_m, uint64_t& acc) {
  uint32_t out;
  asm("{\n\t.reg .b64 x, c, m;\n\t.reg .f32 a, b, sa, sb;\n\t.reg .b16 pa, pb, one;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 c, {%4, %4};\n\t"
      "mov.b64 m, {%5, %5};\n\t"
      "fma.rn.f32x2 x, x, c, m;\n\t"
      "mov.b64 {a, b}, x;\n\t"
      "ex2.approx.ftz.f32 a, a;\n\t"
      "ex2.approx.ftz.f32 b, b;\n\t"
      "cvt.rn.f16x2.f32 %0, b, a;\n\t"
      "mov.b32 {pa, pb}, %0;\n\t"
      "mov.b16 one, 0x3c00;\n\t"
      "mov.b64 {sa, sb}, %1;\n\t"
      "fma.rn.f32.f16 sa, pa, one, sa;\n\t"
      "fma.rn.f32.f16 sb, pb, one, sb;\n\t"
      "mov.b64 %1, {sa, sb};\n\t}"
      : "=r"(out), "+l"(acc)
      : "r"(s0), "r"(s1), "f"(scale), "f"(neg_m));
  return out;
}

// exp2 of an exponent pair, rounded to bf16 and summed as in exp2_pair_bf16.
__device__ __forceinline__ uint32_t exp2_of_pair_bf16(uint64_t x, uint64_t& acc) {
  uint32_t out;
  asm("{\n\t.reg .f32 a, b, sa, sb;\n\t.reg .b16 pa, pb, one;\n\t"
      "mov.b64 {a, b}, %2;\n\t"
      "ex2.approx.ftz.f32 a, a;\n\t"
      "ex2.approx.ftz.f32 b, b;\n\t"
      "cvt.rn.bf16x2.f32 %0, b, a;\n\t"
      "mov.b32 {pa, pb}, %0;\n\t"
      "mov.b16 one, 0x3f80;\n\t"
      "mov.b64 {sa, sb}, %1;\n\t"
      "fma.rn.f32.bf16 sa, pa, one, sa;\n\t"
      "fma.rn.f32.bf16 sb, pb, one, sb;\n\t"
      "mov.b64 %1, {sa, sb};\n\t}"
      : "=r"(out), "+l"(acc)
      : "l"(x));
  return out;
}

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Maximum of three floats in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two-lane fp32 arithmetic on register pairs.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void unpack2u(uint64_t x, uint32_t& a, uint32_t& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// s P(s^2) + c for two raw scores.
template <int N>
__device__ __forceinline__ uint64_t capped_pair(uint32_t s0, uint32_t s1, const float (&poly)[N], uint64_t c) {
  const uint64_t s = pack2u(s0, s1);
  const uint64_t y = mul2(s, s);
  uint64_t t = pack2(poly[N - 1], poly[N - 1]);
#pragma unroll
  for (int i = N - 2; i >= 0; --i) t = fma2(t, y, pack2(poly[i], poly[i]));
  return fma2(s, t, c);
}

// Caps the raw scores of one row and 64 consecutive keys (r) in place, into the
// exp2 domain.  The polynomials hold for the whole warp's scores or not at all.
// No cap (a bias at a scale outside raw_bias_scale): the domain alone.
__device__ __forceinline__ void cap_scores(const TcParams& p, uint32_t* r) {
  float mx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 64; e += 8) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      mx[u] = max3(mx[u], fabsf(__uint_as_float(r[e + 2 * u])), fabsf(__uint_as_float(r[e + 2 * u + 1])));
  }
  const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
  if (!__any_sync(0xffffffffu, top > p.tanh_poly.near_limit)) {
#pragma unroll
    for (int e = 0; e < 64; e += 2) unpack2u(capped_pair(r[e], r[e + 1], p.tanh_poly.near, 0ull), r[e], r[e + 1]);
  } else if (!__any_sync(0xffffffffu, top > p.tanh_poly.wide_limit)) {
#pragma unroll
    for (int e = 0; e < 64; e += 2) unpack2u(capped_pair(r[e], r[e + 1], p.tanh_poly.wide, 0ull), r[e], r[e + 1]);
  } else if (p.mod.cap_log2 == 0.f) {  // (both limits are -infinity then)
#pragma unroll
    for (int e = 0; e < 64; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * p.scale_log2);
  } else if (p.mod.cap_log2 <= kAbsCapLog2) {
#pragma unroll
    for (int e = 0; e < 64; ++e)
      r[e] = __float_as_uint(p.mod.cap_log2 * tanh_by_exp_abs(__uint_as_float(r[e]) * p.mod.raw_to_x));
  } else {
#pragma unroll
    for (int e = 0; e < 64; ++e)
      r[e] = __float_as_uint(p.mod.cap_log2 * tanh_by_exp(__uint_as_float(r[e]) * p.mod.raw_to_x));
  }
}

// Adds the distance bias to the scores of one row and 64 consecutive keys (r),
// in place, one fma per score: `slope` is the bias per key in the scores' units
// (raw, slope / scale, or the exp2 domain after a cap).  dist0 = first key - the
// row's position (distances are whole numbers, so exact); `ahead`: some key may
// lie past the position (a prefix, or full attention), so the distance's absolute
// value is taken.
__device__ __forceinline__ void bias_scores(uint32_t* r, float slope, int dist0, bool ahead) {
  const float d0 = static_cast<float>(dist0);
  if (ahead) {
#pragma unroll
    for (int e = 0; e < 64; ++e)
      r[e] = __float_as_uint(fmaf(-slope, fabsf(d0 + static_cast<float>(e)), __uint_as_float(r[e])));
  } else {
    const uint64_t s2 = pack2(slope, slope), step = pack2(2.f, 2.f);
    uint64_t d = pack2(d0, d0 + 1.f);
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
      unpack2u(fma2(s2, d, pack2u(r[e], r[e + 1])), r[e], r[e + 1]);
      d = add2(d, step);
    }
  }
}

// A value the warp's lanes agree on, told to the compiler as such (it can then live in
// a uniform register and leaves the 96 per thread alone).  The plain form takes it only
// where it spills without (head_dim 128, G = 1: a batch of 16 chunks 39.1 us without, 37.7
// with; the other groups and head_dim 64 run 0.2 to 1.5 % slower with it, the 16k history
// at head_dim 64 4 %).
template <int G, int D, Form kForm>
__device__ __forceinline__ int warp_uniform(int v) {
  if constexpr (kForm == kPlain && !(G == 1 && D == 128)) return v;
  return __shfl_sync(0xffffffffu, v, 0);
}

template <int G, int D, Form kForm>
__global__ void __launch_bounds__(threads(kForm), 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const TcParams p) {
  pdl_enter();
  constexpr int TQ = kBM / G;
  constexpr int kD = D;
  constexpr int kSlabs = Geo<D>::kSlabs;
  constexpr uint32_t kTileQ = Geo<D>::kTileQ;
  constexpr uint32_t kTileKV = Geo<D>::kTileKV;
  constexpr size_t kRecordBytes = Geo<D>::kRecordBytes;
  constexpr bool kFp8 = kForm == kE4m3;
  constexpr bool kQ4 = kForm == kInt4;
  constexpr bool kF16 = quantized(kForm);
  constexpr bool kMod = kForm != kPlain && !kF16;
  constexpr bool kCap = kForm == kCapped || kForm == kCappedBiased;
  constexpr bool kBias = kForm == kBiased || kForm == kCappedBiased;
  // blocks launch in linear order: x runs over (sequence, KV head), y over
  // query-tile pairs from the last (most keys under the causal mask) to the
  // first, and, with a workspace, over the key-range parts of each pair
  const int seq = blockIdx.x / p.hkv;
  const int g = blockIdx.x % p.hkv;
  const int pairs = p.q_tiles / 2;
  const int pt = pairs - 1 - static_cast<int>(blockIdx.y) / p.parts_max;
  const int part = static_cast<int>(blockIdx.y) % p.parts_max;
  const int q_begin = warp_uniform<G, D, kForm>(__ldg(p.cu_q + seq));
  const int nq = warp_uniform<G, D, kForm>(__ldg(p.cu_q + seq + 1)) - q_begin;
  const int k_begin = warp_uniform<G, D, kForm>(__ldg(p.cu_k + seq));
  const int nk = warp_uniform<G, D, kForm>(__ldg(p.cu_k + seq + 1)) - k_begin;
  // cu_seqlens must describe rows inside q / out (and the packed k / v), and no
  // sequence may have more rows than max_seqlen_q, which sized the grid: such a
  // sequence is skipped whole and raises the range bit
  if (q_begin < 0 || nq < 0 || nk < nq || static_cast<long long>(q_begin) + nq > p.total_q || nq > p.max_seqlen_q ||
      (p.paged ? static_cast<long long>(nk) > static_cast<long long>(p.max_blocks) * p.block_size
               : (k_begin < 0 || static_cast<long long>(k_begin) + nk > p.total_k))) {
    if (threadIdx.x == 0) raise_error(p.err, PKV_DERR_LEN_RANGE);
    return;
  }
  const int tok0 = pt * 2 * TQ;  // first token of tile A; tile B starts TQ later
  if (tok0 >= nq) return;
  const int cached = nk - nq;
  // kMod: keys below prefix_end are visible to every row besides the causal ones;
  // no row of the pair sees a key before lo_pair
  int prefix_end = 0;
  int lo_pair = 0;
  if constexpr (kMod) {
    if (p.mod.prefix_lens) prefix_end = warp_uniform<G, D, kForm>(min(max(__ldg(p.mod.prefix_lens + seq), 0), nk));
    if (p.mod.first_keys) {
      int least = INT32_MAX;
      for (int t = tok0 + static_cast<int>(threadIdx.x % 32); t < min(nq, tok0 + 2 * TQ); t += 32)
        least = min(least, __ldg(p.mod.first_keys + q_begin + t));
      lo_pair = max(__reduce_min_sync(0xffffffffu, least), 0);
    }
  }
  // key tiles up to the last one each query tile needs (0: the tile has no rows)
  int n_need[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int t0 = tok0 + x * TQ;
    int keys = t0 >= nq ? 0 : (p.causal ? cached + min(nq, t0 + TQ) : nk);
    if constexpr (kMod) {
      if (t0 < nq) keys = max(keys, prefix_end);
      if (keys <= lo_pair) keys = 0;  // no row of the tile sees a key
    }
    n_need[x] = (keys + kBN - 1) / kBN;
  }
  int j_first = 0;  // the pair's first key tile
  if constexpr (kMod) j_first = min(lo_pair / kBN, max(n_need[0], n_need[1]));
  const int n_all = max(n_need[0], n_need[1]) - j_first;
  // this CTA's key tiles: j0 .. j0 + n_tiles - 1 (all of them, or one of up to P
  // consecutive ranges); tile X takes the first n_x of them
  const int parts = n_all > kSplitMinTiles ? min(p.parts_max, (n_all + kSplitMinTiles - 1) / kSplitMinTiles) : 1;
  if (part >= parts) return;
  const int j0 = j_first + part * n_all / parts;
  const int n_tiles = j_first + (part + 1) * n_all / parts - j0;
  const int n_a = max(0, min(n_tiles, n_need[0] - j0));
  const int n_b = max(0, min(n_tiles, n_need[1] - j0));
  // the last tile holds keys past nk: its V rows there are zeroed first
  // (kFp8, kInt4: the widening warps write those rows as zeros)
  const bool v_tail = !kF16 && (!kMod || n_tiles > 0) && (j0 + n_tiles) * kBN > nk;
  // kMod: the first tile holds keys before lo_pair: its V rows there are zeroed too
  const bool v_head = kMod && n_tiles > 0 && j0 * kBN < lo_pair;

  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char* sq = smem;  // Q_A, then Q_B
  unsigned char* sk = sq + 2 * kTileQ;
  unsigned char* sv = sk + kStages * kTileKV;
  float* red = reinterpret_cast<float*>(smem + Geo<D>::kRedOffset);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Geo<D>::kBarOffset);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_ticket = abort_flag + 1;  // split tiles' tickets, one per query tile

  const int tid = threadIdx.x;
  const int warp = warp_uniform<G, D, kForm>(tid / 32);
  const int lane = tid % 32;
  const int32_t* table = p.block_tables + static_cast<size_t>(seq) * p.max_blocks;

  if (tid == 0) {
    *abort_flag = 0;
    mbar_init(&bars[Q_FULL], 1);
    for (int s = 0; s < kStages; ++s) {
      // kFp8: one arrival per widening warp, kInt4: per quarter
      mbar_init(&bars[K_FULL + s], kFp8 ? kWidenWarps : kQ4 ? kBN / kQuarter : 1);
      mbar_init(&bars[V_FULL + s], kFp8 ? kWidenWarps : kQ4 ? kBN / kQuarter : 1);
      mbar_init(&bars[K_EMPTY + s], 1);
      mbar_init(&bars[V_EMPTY + s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars[S_FULL + x], 1);
      mbar_init(&bars[P_FULL + x], kSoftmaxWarps);  // one arrival per softmax warp
    }
    mbar_init(&bars[O_FINAL], 1);
    mbar_init(&bars[O_FINAL + 1], 1);
    mbar_init(&bars[V_TAIL], 1);
    if constexpr (kMod) mbar_init(&bars[V_HEAD], 1);
    if constexpr (kF16) {
      for (int x = 0; x < 2; ++x) mbar_init(&bars[Q_READY + x], kSoftmaxWarps);
      for (int s = 0; s < 2 * kStages; ++s) mbar_init(&bars[RAW_FULL + s], 1);
    }
    fence_mbar_init();
  }
  const Waiter wait{abort_flag, p.err};
  // kFp8: where the codes of row r of a tile lie in its stage
  auto raw_offset = [](int r) -> uint32_t {
    return D == 128 ? kSlabKV + r * 128 : (r / kQuarter) * (kQuarter * 128) + kQuarter * 64 + (r % kQuarter) * 64;
  };
  // Loads tile j's K (is_v = false) or V into stage j % kStages, after the
  // stage's previous occupant (tile j - kStages) was released.  One thread issues
  // the plain kernel's copies; the other forms' the whole warp, a piece per lane
  // (block sizes that share few factors of 2 with 128 make many pieces).  kFp8:
  // the codes of each quarter go to the end of its own part of the stage, which the
  // widened rows then take: at head_dim 128 the rows of the second slab, at 64 the
  // second half of the quarter's rows.
  auto load_tile = [&](int j, bool is_v) {
    const int st = j % kStages;
    const int use = j / kStages;
    uint64_t* full = &bars[(is_v ? V_FULL : K_FULL) + st];
    if (use > 0) wait(&bars[(is_v ? V_EMPTY : K_EMPTY) + st], (use - 1) & 1);
    unsigned char* dst = (is_v ? sv : sk) + st * kTileKV;
    const CUtensorMap* map = is_v ? &tm_v : &tm_k;
    const int key0 = (j0 + j) * kBN;
    if constexpr (kFp8) {
      __syncwarp();
      uint64_t* raw_full = &bars[RAW_FULL + (is_v ? kStages : 0) + st];
      for (int r = lane * p.piece_rows; r < kBN; r += 32 * p.piece_rows) {
        const int key = key0 + r;
        if (key >= nk) continue;
        const int blk = key / p.block_size;
        const int phys = __ldg(table + blk);
        if (phys < 0 || phys >= p.num_blocks) {
          raise_error(p.err, PKV_DERR_BLOCK_RANGE);
          continue;
        }
        const int row = phys * p.block_size + (key - blk * p.block_size);
        unsigned char* to = dst + raw_offset(r);
        mbar_expect_tx(raw_full, p.piece_rows * D);
        if (p.piece_rows > 1)
          tc::tma_load_3d(to, map, 0, g, row, raw_full);
        else  // a tensor copy of one 64-byte row could start off its 128-byte boundary
          bulk_g2s(to, (is_v ? p.v_codes : p.k_codes) + (static_cast<size_t>(row) * p.hkv + g) * D, D, raw_full,
                   l2_normal_policy());
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(raw_full);
      return;
    }
    if constexpr (kMod) {
      __syncwarp();
      const int piece = p.paged ? p.piece_rows : kBN;
      const uint32_t piece_bytes = piece * 128u;
      for (int r = lane * piece; r < kBN; r += 32 * piece) {
        const int key = key0 + r;
        if (key >= nk || key + piece <= lo_pair) continue;
        int row = k_begin + key;
        if (p.paged) {
          const int blk = key / p.block_size;
          const int phys = __ldg(table + blk);
          if (phys < 0 || phys >= p.num_blocks) {
            raise_error(p.err, PKV_DERR_BLOCK_RANGE);
            continue;
          }
          row = phys * p.block_size + (key - blk * p.block_size);
        }
        mbar_expect_tx(full, kSlabs * piece_bytes);
        tc::tma_load_3d(dst + r * 128, map, 0, g, row, full);
        if constexpr (kSlabs == 2) tc::tma_load_3d(dst + kSlabKV + r * 128, map, 64, g, row, full);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
      return;
    }
    if (p.paged) {
      const uint32_t piece_bytes = p.piece_rows * 128u;
      for (int r = 0; r < kBN; r += p.piece_rows) {
        const int key = key0 + r;
        if (key >= nk) break;
        const int blk = key / p.block_size;
        const int phys = __ldg(table + blk);
        if (phys < 0 || phys >= p.num_blocks) {
          raise_error(p.err, PKV_DERR_BLOCK_RANGE);
          continue;
        }
        const int row = phys * p.block_size + (key - blk * p.block_size);
        mbar_expect_tx(full, kSlabs * piece_bytes);
        tc::tma_load_3d(dst + r * 128, map, 0, g, row, full);
        if constexpr (kSlabs == 2) tc::tma_load_3d(dst + kSlabKV + r * 128, map, 64, g, row, full);
      }
    } else {
      const int row = k_begin + key0;
      mbar_expect_tx(full, kTileKV);
      tc::tma_load_3d(dst, map, 0, g, row, full);
      if constexpr (kSlabs == 2) tc::tma_load_3d(dst + kSlabKV, map, 64, g, row, full);
    }
    mbar_arrive(full);
  };
  // the producer thread issues Q and the first K/V tiles (stages still free)
  // before the CTA-wide sync, so their latency overlaps the TMEM allocation
  const int n_early = min(n_tiles, kStages);
  if (tid == 0) {
    tc::prefetch_tensormap(&tm_q);
    if constexpr (!kQ4) {
      tc::prefetch_tensormap(&tm_k);
      tc::prefetch_tensormap(&tm_v);
    }
    const int nx = n_b > 0 ? 2 : 1;
    mbar_expect_tx(&bars[Q_FULL], nx * kTileQ);
    for (int x = 0; x < nx; ++x) {
      tc::tma_load_3d(sq + x * kTileQ, &tm_q, 0, g * G, q_begin + tok0 + x * TQ, &bars[Q_FULL]);
      if constexpr (kSlabs == 2)
        tc::tma_load_3d(sq + x * kTileQ + kSlabQ, &tm_q, 64, g * G, q_begin + tok0 + x * TQ, &bars[Q_FULL]);
    }
    mbar_arrive(&bars[Q_FULL]);
    if constexpr (!kMod && !kF16) {
      for (int j = 0; j < n_early; ++j) {
        load_tile(j, false);
        load_tile(j, true);
      }
    }
  }
  if constexpr (kMod || kFp8) {
    if (warp == 0) {
      __syncwarp();  // the barriers are initialised
      for (int j = 0; j < n_early; ++j) {
        load_tile(j, false);
        load_tile(j, true);
      }
    }
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // broadcast from lane 0 so the compiler treats the TMEM base as warp-uniform
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (kQ4 && (warp == 0 || warp >= 2 + 2 * kSoftmaxWarps)) {
    // ------------------------------------------------------------ kInt4: rows to f16
    // The quarters of K(0), V(0), K(1), ... go round the three warps.
    constexpr int kWorkers = kWidenWarps + 1;
    constexpr int kChunks = D / 32;  // 16-byte chunks of a head's codes: 32 elements, 4 chunks of the f16 row
    const int me = warp == 0 ? 0 : warp - 1 - 2 * kSoftmaxWarps;
    const int n_units = 8 * n_tiles;
    const int row_bytes = q4_row_bytes(p.hkv, D);
    const int scale_at = q4_scale_offset(p.hkv, D) + g * (D / 16);
    unsigned char* const ring = smem + Geo<D>::kInt4Offset + me * (kInt4Depth * Geo<D>::kInt4Slot);
    // the block of this lane's key of a unit (-1: no such key) is looked up a unit before its copy
    auto key_of = [&](int u) { return (j0 + (u >> 3)) * kBN + (u & 3) * kQuarter + lane; };
    auto block_of = [&](int key) {
      return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(key)) * p.block_mul >> p.block_shift);
    };
    // where chunk ch of row r lies in the ring: eight rows' same chunks (and eight neighbouring chunks) differ modulo 128 bytes
    auto swizzle = [](int r) { return kChunks == 4 ? (r >> 1) & 3 : (r >> 2) & 1; };
    int phys = -1, in_block = 0;
    auto look_up = [&](int u) {
      const int key = key_of(u);
      phys = -1;
      if (u < n_units && key < nk) {
        const int blk = block_of(key);
        in_block = key - blk * p.block_size;
        phys = __ldg(table + blk);
      }
    };
    look_up(me);
    int slot = 0;  // of the next unit to copy
    // rows of no key and of bad blocks are filled with zeros
    auto copy = [&](int u) {
      if (u < n_units) {
        const bool ok = phys >= 0 && phys < p.num_blocks;
        if (!ok && key_of(u) < nk) raise_error(p.err, PKV_DERR_BLOCK_RANGE);
        const int row = ok ? phys * p.block_size + in_block : -1;
        const unsigned char* pool = u & 4 ? p.v_codes : p.k_codes;
        const uint32_t to = smem_u32(ring + slot * Geo<D>::kInt4Slot);
        // neighbouring lanes take the chunks of one row
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int r = i * (32 / kChunks) + lane / kChunks;
          const int from = __shfl_sync(0xffffffffu, row, r);
          const int ch = lane % kChunks;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (r * kChunks + (ch ^ swizzle(r))) * 16),
                       "l"(pool + static_cast<size_t>(max(from, 0)) * row_bytes + g * (D / 2) + ch * 16),
                       "r"(from >= 0 ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to + Geo<D>::kInt4Codes + lane * (D / 16)),
                     "l"(pool + static_cast<size_t>(max(row, 0)) * row_bytes + scale_at), "n"(D / 16),
                     "r"(row >= 0 ? D / 16 : 0)
                     : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      look_up(u + kWorkers);
      slot = slot + 1 == kInt4Depth ? 0 : slot + 1;
    };
#pragma unroll
    for (int i = 0; i < kInt4Depth - 1; ++i) copy(me + i * kWorkers);
    int from = 0;
    for (int u = me; u < n_units; u += kWorkers) {
      copy(u + (kInt4Depth - 1) * kWorkers);
      asm volatile("cp.async.wait_group %0;" ::"n"(kInt4Depth - 1) : "memory");
      __syncwarp();
      const unsigned char* src = ring + from * Geo<D>::kInt4Slot;
      from = from + 1 == kInt4Depth ? 0 : from + 1;
      uint4 codes[kChunks];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) codes[i] = lds128(src + (lane * kChunks + (i ^ swizzle(lane))) * 16);
      uint32_t scales[D / 64];  // E4M3, four groups each
      if constexpr (D == 128) {
        const uint2 x = *reinterpret_cast<const uint2*>(src + Geo<D>::kInt4Codes + lane * 8);
        scales[0] = x.x, scales[1] = x.y;
      } else {
        scales[0] = *reinterpret_cast<const uint32_t*>(src + Geo<D>::kInt4Codes + lane * 4);
      }
      const int j = u >> 3;
      const bool is_v = u & 4;
      const int st = j % kStages;
      if (j >= kStages) wait(&bars[(is_v ? V_EMPTY : K_EMPTY) + st], (j / kStages - 1) & 1);
      const int row = (u & 3) * kQuarter + lane;
      unsigned char* dst = (is_v ? sv : sk) + st * kTileKV + row * 128;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
        // the chunk's two groups: bytes 2 i and 2 i + 1 of the scales
        const uint32_t s = e4m3x2_to_f16x2(scales[i / 2] >> (16 * (i & 1)) & 0xffffu);
        const Q4Scale k[2] = {Q4Scale(prmt(s, 0, 0x1010u)), Q4Scale(prmt(s, 0, 0x3232u))};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t f[4];
          widen_q4(w[e], k[e / 2], f);
          const int ch = 4 * i + e;
          *reinterpret_cast<uint4*>(dst + (ch >> 3) * kSlabKV + (((ch & 7) ^ (row & 7)) << 4)) =
              make_uint4(f[0], f[1], f[2], f[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[(is_v ? V_FULL : K_FULL) + st]);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // V rows of tile j's stage from row `first` on, `count` of them, become zeros once the tile has arrived
    auto zero_v_rows = [&](int j, int first, int count) {
      const int st = j % kStages;
      wait(&bars[V_FULL + st], (j / kStages) & 1);
      unsigned char* vt = sv + st * kTileKV;
      for (int idx = lane; idx < count * kSlabs * 8; idx += 32) {
        const int rr = first + idx / (kSlabs * 8);
        const int ch = idx % (kSlabs * 8);
        *reinterpret_cast<uint4*>(vt + (ch >> 3) * kSlabKV + rr * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    if constexpr (kFp8) {
      if (parts > 1 && p.piece_rows > 1) {  // as below
        for (int key = (j0 + n_early) * kBN + lane * p.piece_rows; key < min((j0 + n_tiles) * kBN, nk);
             key += 32 * p.piece_rows) {
          const int blk = key / p.block_size;
          const int phys = __ldg(table + blk);
          if (phys < 0 || phys >= p.num_blocks) continue;  // raised by the load
          const int row = phys * p.block_size + (key - blk * p.block_size);
          tc::tma_prefetch_3d(&tm_k, 0, g, row);
          tc::tma_prefetch_3d(&tm_v, 0, g, row);
        }
        __syncwarp();
      }
      for (int j = n_early; j < n_tiles; ++j) {
        load_tile(j, false);
        load_tile(j, true);
      }
    } else if constexpr (kMod) {
      if (parts > 1) {
        // a split part streams a key range no other CTA reads: request it into
        // L2 first, a piece per lane
        const int piece = p.paged ? p.piece_rows : kBN;
        for (int key = (j0 + n_early) * kBN + lane * piece; key < min((j0 + n_tiles) * kBN, nk); key += 32 * piece) {
          if (key + piece <= lo_pair) continue;
          int row = k_begin + key;
          if (p.paged) {
            const int blk = key / p.block_size;
            const int phys = __ldg(table + blk);
            if (phys < 0 || phys >= p.num_blocks) continue;  // raised by the load
            row = phys * p.block_size + (key - blk * p.block_size);
          }
          tc::tma_prefetch_3d(&tm_k, 0, g, row);
          if constexpr (kSlabs == 2) tc::tma_prefetch_3d(&tm_k, 64, g, row);
          tc::tma_prefetch_3d(&tm_v, 0, g, row);
          if constexpr (kSlabs == 2) tc::tma_prefetch_3d(&tm_v, 64, g, row);
        }
        __syncwarp();
      }
      if (v_head) {
        // rows before lo_pair (of blocks not read, or of keys that no row of the pair sees)
        zero_v_rows(0, 0, lo_pair - j0 * kBN);
        if (lane == 0) mbar_arrive(&bars[V_HEAD]);
      }
      for (int j = n_early; j < n_tiles; ++j) {
        load_tile(j, false);
        load_tile(j, true);
      }
    } else if (lane == 0) {
      if (parts > 1) {
        // a split part streams a key range no other CTA reads: request it into
        // L2 first, so that the ring's loads, which start only as stages free
        // up, find it there
        for (int j = n_early; j < n_tiles; ++j) {
          const int key0 = (j0 + j) * kBN;
          for (int r = 0; r < kBN; r += p.piece_rows) {
            const int key = key0 + r;
            if (key >= nk) break;
            int row = k_begin + key;
            if (p.paged) {
              const int blk = key / p.block_size;
              const int phys = __ldg(table + blk);
              if (phys < 0 || phys >= p.num_blocks) continue;  // raised by the load
              row = phys * p.block_size + (key - blk * p.block_size);
            }
            tc::tma_prefetch_3d(&tm_k, 0, g, row);
            if constexpr (kSlabs == 2) tc::tma_prefetch_3d(&tm_k, 64, g, row);
            tc::tma_prefetch_3d(&tm_v, 0, g, row);
            if constexpr (kSlabs == 2) tc::tma_prefetch_3d(&tm_v, 64, g, row);
          }
        }
      }
      // K(j) once the K stage is free (both Q K^T of tile j - 2 read it), V(j)
      // once the V stage is
      for (int j = n_early; j < n_tiles; ++j) {
        load_tile(j, false);
        load_tile(j, true);
      }
    }
    __syncwarp();  // every load issued before the warp turns to the last tile
    if (v_tail) {
      // In the last tile the V rows past nk hold whatever their block had there
      // (or were not loaded): zero them so 0 * stale never reaches O.  Every
      // load has been issued, so the stage's barrier is at the last tile's
      // phase or just past it, and a parity wait for that phase is exact.
      zero_v_rows(n_tiles - 1, nk - (j0 + n_tiles - 1) * kBN, (j0 + n_tiles) * kBN - nk);
      if (lane == 0) mbar_arrive(&bars[V_TAIL]);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop (its descriptor arithmetic stays warp-uniform);
    // one elected lane issues the MMAs and commits.
    {
      const bool leader = tc::elect_one();
      constexpr uint32_t idesc_qk = kF16 ? tc::idesc_f16(kBM, kBN, 0, 0) : tc::idesc_bf16(kBM, kBN, 0, 0);
      constexpr uint32_t idesc_pv = kF16 ? tc::idesc_f16(kBM, kD, 0, 1) : tc::idesc_bf16(kBM, kD, 0, 1);
      // descriptors of the first Q, K and V slabs; later ones differ only in the
      // start-address field (address >> 4), so they are reached by adding offset >> 4
      const uint64_t q_desc = tc::smem_desc(smem_u32(sq), 16, 1024);
      const uint64_t k_desc = tc::smem_desc(smem_u32(sk), 16, 1024);
      const uint64_t v_desc = tc::smem_desc(smem_u32(sv), kSlabKV, 1024);
      const int n_x[2] = {n_a, n_b};
      // S_X = Q_X K(j)^T (S_X held P_X(j - 1), read by P_X(j - 1) V issued
      // before: the tensor pipe runs one thread's MMAs in order)
      auto issue_qk = [&](int x, int j) {
        const int st = j % kStages;
        // the chain's first step: tile X's Q slab 0 and stage st's K slab 0
        const uint64_t a0 = q_desc + ((x * kTileQ) >> 4);
        const uint64_t b0 = k_desc + ((st * kTileKV) >> 4);
        if (leader) {
          if constexpr (kD == 128)
            tc::mma_ss_k128(tmem + kColS + x * kBN, a0, b0, idesc_qk);
          else
            tc::mma_ss_k64(tmem + kColS + x * kBN, a0, b0, idesc_qk);
        }
        if (leader) tc::commit(&bars[S_FULL + x]);
      };
      // O_X += P_X(j) V(j)
      auto issue_pv = [&](int x, int j) {
        const int st = j % kStages;
        wait.ready(&bars[P_FULL + x], j & 1);
        tc::fence_after_sync();
        if (leader)
          tc::mma_ts_k128(tmem + kColO + x * kD, tmem + kColS + x * kBN, v_desc + ((st * kTileKV) >> 4), idesc_pv,
                          j > 0 ? 1u : 0u);
      };
      wait(&bars[Q_FULL], 0);
      if (n_tiles > 0) {
        wait.ready(&bars[K_FULL], 0);
        tc::fence_after_sync();
        for (int x = 0; x < 2; ++x)
          if (n_x[x] > 0) {
            if constexpr (kF16) {
              wait(&bars[Q_READY + x], 0);
              tc::fence_after_sync();
            }
            issue_qk(x, 0);
          }
        if (leader) tc::commit(&bars[K_EMPTY]);
      }
      for (int x = 0; x < 2; ++x)
        if (leader && (n_x[x] == 0)) tc::commit(&bars[O_FINAL + x]);  // a tile with no key tile here: nothing to wait for
      for (int j = 0; j < n_tiles; ++j) {
        const int st = j % kStages;
        if constexpr (kMod) {
          if (v_head && j == 0) wait(&bars[V_HEAD], 0);
        }
        if (v_tail && j == n_tiles - 1)
          wait(&bars[V_TAIL], 0);
        else
          wait.ready(&bars[V_FULL + st], (j / kStages) & 1);
        const bool next = j + 1 < n_tiles;
        bool k_next = false;  // K(j + 1) seen loaded
        for (int x = 0; x < 2; ++x) {
          if (j < n_x[x]) {
            issue_pv(x, j);
            if (leader && (j == n_x[x] - 1)) tc::commit(&bars[O_FINAL + x]);
            // the step's last P V (tile B's, or A's when B has no tile j) releases V(j)
            if (leader && (x == 1 || j >= n_x[1])) tc::commit(&bars[V_EMPTY + st]);
          }
          if (j + 1 < n_x[x]) {
            if (!k_next) {
              wait.ready(&bars[K_FULL + (j + 1) % kStages], ((j + 1) / kStages) & 1);
              tc::fence_after_sync();
              k_next = true;
            }
            issue_qk(x, j + 1);
          }
        }
        if (leader && next) tc::commit(&bars[K_EMPTY + (j + 1) % kStages]);
      }
      // no MMA may be in flight when TMEM is freed: tile B's last product (or
      // A's, when B has none here) is the last MMA issued
      wait(&bars[O_FINAL + (n_b > 0 ? 1 : 0)], 0);
    }
  } else if (kFp8 && warp >= 2 + 2 * kSoftmaxWarps) {
    // ------------------------------------------------------------ kFp8: widen codes to f16
    // Each warp takes two quarters of every tile: a quarter's codes go to registers,
    // then their f16 rows over them.  Sixteen codes (one 16-byte chunk) become two
    // chunks of the swizzled f16 row.  A group of eight lanes takes two
    // neighbouring rows, at head_dim 128 from opposite slabs: its loads cover 128
    // distinct bytes modulo 128, and its stores the even chunk positions of one row
    // and the odd ones of the other, so neither has bank conflicts.
    constexpr int kIter = D / 16;
    const int me = warp - 2 - 2 * kSoftmaxWarps;
    const int odd = (lane >> 2) & 1;
    const int row0 = 2 * (lane >> 3) + odd;  // in the quarter; + 8 per two (head_dim 128) or one iterations
    const uint32_t at0 = ((2 * (lane & 3)) ^ (row0 & 7)) << 4;
    for (int n = 0; n < 2 * n_tiles; ++n) {
      const int j = n >> 1;
      const bool is_v = n & 1;
      const int st = j % kStages;
      unsigned char* stage = (is_v ? sv : sk) + st * kTileKV;
      wait(&bars[RAW_FULL + (is_v ? kStages : 0) + st], (j / kStages) & 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int first = (2 * me + h) * kQuarter;  // first row of the quarter
        const unsigned char* raw = stage + raw_offset(first) + row0 * D + (lane & 3) * 16;
        uint4 codes[kIter];
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          if constexpr (D == 128)
            codes[i] = lds128(raw + (i >> 1) * 8 * D + ((i & 1) ^ odd) * 64);
          else
            codes[i] = lds128(raw + i * 8 * D);
        }
        __syncwarp();  // every code of the quarter is in registers
        unsigned char* dst = stage + (first + row0) * 128 + at0;
        const int rows = nk - (j0 + j) * kBN - first - row0;  // row0 + i of the quarter holds a key: i < rows
        auto widen = [&](bool partial) {
#pragma unroll
          for (int i = 0; i < kIter; ++i) {
            const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
            uint32_t f[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) e4m3x4_to_f16x4(w[u], f[2 * u], f[2 * u + 1]);
            const int step = D == 128 ? (i >> 1) * 8 : i * 8;
            if (partial && step >= rows) {  // past the last key: whatever the stage held
#pragma unroll
              for (int u = 0; u < 8; ++u) f[u] = 0u;
            }
            unsigned char* to = dst + step * 128 + (D == 128 ? ((i & 1) ^ odd) * kSlabKV : 0);
            *reinterpret_cast<uint4*>(to) = make_uint4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<uint4*>(to + (at0 & 16 ? -16 : 16)) = make_uint4(f[4], f[5], f[6], f[7]);
          }
        };
        if (nk >= (j0 + j) * kBN + first + kQuarter)
          widen(false);
        else
          widen(true);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[(is_v ? V_FULL : K_FULL) + st]);
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue of tile X, one half of the keys
    const int x = (warp - 2) / kSoftmaxWarps;
    const int half = ((warp - 2) % kSoftmaxWarps) / 4;
    const int n_x = x == 0 ? n_a : n_b;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const int gt = half * kBM + row;  // 0..255 within the tile's softmax threads
    const int tok_first = tok0 + x * TQ;  // first token of this query tile
    const int tok = tok_first + row / G;
    const int pos = cached + tok;  // absolute position of this query row
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_addr = lane_addr + kColS + x * kBN;
    const uint32_t o_addr = lane_addr + kColO + x * kD + half * (kD / 2);  // this half's D / 2 output columns
    const int lim = p.causal ? min(pos, nk - 1) : nk - 1;
    // kMod: the row sees keys lo .. hi; a row that sees none gets a range no key is
    // in.  Taken anew for each tile that needs it: held through the loop, the two
    // would cost registers.  Rows past the last token see none: a warp's rows share the
    // decision to rescale, and such a row's scores of keys that were not read (stale
    // shared memory) would change the other rows' rounding from run to run.
    auto seen_range = [&](int& lo, int& hi) {
      hi = max(lim, prefix_end - 1);
      lo = p.mod.first_keys && tok < nq ? max(__ldg(p.mod.first_keys + q_begin + tok), 0) : 0;
      if (lo > hi || tok >= nq) lo = hi = INT32_MAX;
    };
    int lo_most = 0;     // the largest lo of the warp
    float slope = 0.f;   // per key of distance, in the units of bias_scores
    if constexpr (kMod) {
      int hi;
      seen_range(lo_most, hi);
      lo_most = __reduce_max_sync(0xffffffffu, tok < nq ? lo_most : 0);
      if constexpr (kBias) slope = __ldg(p.mod.slopes + g * G + row % G) * p.bias_mul;
    }
    float mul = kBias && kCap ? 1.f : p.scale_log2;  // scores as held in registers to exponents
    const int bar_id = 1 + x;                 // the tile's 8 softmax warps
    const int pair_id = 3 + x * 4 + quad;     // the tile's two warps (one per half) on these 32 rows
    constexpr int kGroup = 32 * kSoftmaxWarps;
    auto red_at = [&](int parity, int h) { return red + ((parity * 2 + x) * 2 + h) * kBM + row; };
    float m_run = -INFINITY;
    float l_run = 0.f;  // this half's keys only
    bool large = false;  // kF16: a row of the warp has a reference of 2^20 or more
    uint32_t r[64];
    if constexpr (kF16) {
      // Q becomes f16 in place, each row scaled by the power of two that puts its
      // largest element in [2^14, 2^15): exact but for elements 2^28 times
      // smaller than that.  The power comes off with the softmax scale.
      int ex = 0;
      if (n_x > 0) {
        // tile A first: its products can start while B's rows are rewritten
        wait(&bars[x == 1 && n_a > 0 ? Q_READY : Q_FULL], 0);
        if (x == 1) wait(&bars[Q_FULL], 0);
        constexpr int kChunksHalf = D / 16;  // this half's 16-byte chunks of the row
        unsigned char* q_row = sq + x * kTileQ + (D == 128 ? half * kSlabQ : 0) + row * 128;
        auto q_chunk = [&](int i) {
          const int ch = D == 128 ? i : half * kChunksHalf + i;
          return reinterpret_cast<uint4*>(q_row + ((ch ^ (row & 7)) << 4));
        };
        uint32_t top2 = 0u;  // a bf16 pair: the largest magnitudes of even and odd columns
        uint4 qc[kChunksHalf];
#pragma unroll
        for (int i = 0; i < kChunksHalf; ++i) {
          qc[i] = *q_chunk(i);
          const uint32_t w[4] = {qc[i].x, qc[i].y, qc[i].z, qc[i].w};
#pragma unroll
          for (int u = 0; u < 4; ++u) asm("max.bf16x2 %0, %0, %1;" : "+r"(top2) : "r"(w[u] & 0x7fff7fffu));
        }
        float top = fmaxf(__uint_as_float(top2 << 16), __uint_as_float(top2 & 0xffff0000u));
        *red_at(0, half) = top;
        named_barrier_sync(pair_id, 64);
        top = fmaxf(*red_at(0, 0), *red_at(0, 1));
        const int exponent = static_cast<int>(__float_as_uint(top) >> 23) - 127;  // -127 for zero and subnormals
        ex = min(max(14 - exponent, -113), 126);
        const float up = power_of_two(ex);
#pragma unroll
        for (int i = 0; i < kChunksHalf; ++i) {
          float f[8];
          Chunk<__nv_bfloat16>::unpack(qc[i], f);
          if constexpr (kQ4)
            *q_chunk(i) = make_uint4(pack_f16x2(f[0] * up, f[4] * up), pack_f16x2(f[1] * up, f[5] * up),
                                     pack_f16x2(f[2] * up, f[6] * up), pack_f16x2(f[3] * up, f[7] * up));
          else
            *q_chunk(i) = make_uint4(pack_f16x2(f[0] * up, f[1] * up), pack_f16x2(f[2] * up, f[3] * up),
                                     pack_f16x2(f[4] * up, f[5] * up), pack_f16x2(f[6] * up, f[7] * up));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Q_READY + x]);
      mul = row_scale(mul, p.scale_exp - ex);
    }

    // kMod: keys the row does not see get -infinity; lo <= key <= hi in one unsigned comparison
    bool masked = false;
    auto hide = [&](int key0) {
      int lo, hi;
      seen_range(lo, hi);
      const uint32_t span = static_cast<uint32_t>(hi - lo);
      const uint32_t off = static_cast<uint32_t>(key0 - lo);
#pragma unroll
      for (int e = 0; e < 64; ++e) {
        // (a cap tells a key not seen, -infinity, from a score that overflowed)
        if constexpr (kCap && !kBias) r[e] = __float_as_uint(max_nan(__uint_as_float(r[e]), -FLT_MAX));
        if (off + e > span) r[e] = __float_as_uint(-INFINITY);
      }
    };

    for (int j = 0; j < n_x; ++j) {
      const int key0 = (j0 + j) * kBN + half * 64;  // first key of this half
      wait(&bars[S_FULL + x], j & 1);
      tc::fence_after_sync();
      // this half's 64 scores, held in registers: the other half writes its P
      // over them once both halves have exchanged their maxima
      tc::tmem_ld32(s_addr + half * 64, r);
      tc::tmem_ld32(s_addr + half * 64 + 32, r + 32);
      tc::tmem_wait_ld();
      if constexpr (kMod) {
        const int seen_by_all = p.causal ? max(cached + tok_first, prefix_end - 1) : nk - 1;
        masked = key0 + 63 > seen_by_all || key0 < lo_most;
        if constexpr (kBias && kCap) {
          // the scores' size chooses how the cap is taken: keys that were not read (stale shared memory), or lie past
          // the sequence's end, must not count
          if (key0 < lo_pair || key0 + 63 >= nk) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (key0 + e < lo_pair || key0 + e >= nk) r[e] = 0u;
          }
          cap_scores(p, r);
        }
        if constexpr (kBias) bias_scores(r, slope, key0 - pos, key0 + 63 > cached + tok_first);
        if (masked) hide(key0);
      } else if (key0 + 63 > (p.causal ? cached + tok_first : nk - 1)) {
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (key0 + e > lim) r[e] = __float_as_uint(-INFINITY);
      }
      // raw-score maximum of this half (the scale, > 0, is applied after), as
      // four chains of three-input maxima; then the row's, through shared memory
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 64; e += 8) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          mx[u] = max3(mx[u], __uint_as_float(r[e + 2 * u]), __uint_as_float(r[e + 2 * u + 1]));
      }
      float mx_half = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
      if constexpr (kCap && !kBias) {
        if (!masked) mx_half = fmaxf(mx_half, -FLT_MAX);  // -infinity stands for "sees no key"
      }
      *red_at(j & 1, half) = mx_half;
      named_barrier_sync(pair_id, 64);
      const float mt = fmaxf(*red_at(j & 1, 0), *red_at(j & 1, 1));
      const float top = __fmul_rn(mt, mul);
      // kF16: the reference of the weights is below the maximum; the factor cancels against the row sum and in the
      // merge of parts, which see the same reference
      float m_tile = kF16 ? __fadd_rn(top, -kF16WeightLog2) : top;
      if constexpr (kCap && !kBias) {
        m_tile = mt == -INFINITY ? mt : p.mod.cap_log2 * tanh_by_exp(mt * p.mod.raw_to_x);
      }
      const float m_new = fmaxf(m_run, m_tile);
      // (kF16: the largest exponent itself decides, so that no rounding of a large reference lets a weight pass f16's range)
      const bool grow = kF16 ? top - m_run > kRescaleLog2 + kF16WeightLog2
                             : m_new > m_run + kRescaleLog2 || (m_run == -INFINITY && m_new != -INFINITY);
      const bool rescale = __any_sync(0xffffffffu, grow);  // the same in both halves' warps
      float factor = 1.f;
      if (rescale) {
        factor = (m_run == -INFINITY || m_new <= m_run) ? 1.f : exp2f(m_run - m_new);
        m_run = fmaxf(m_run, m_new);
        // (-infinity, no key yet, is not such a reference)
        if constexpr (kF16) large = __any_sync(0xffffffffu, fabsf(m_run) >= 0x1p20f && m_run != -INFINITY);
      }
      const float m_use = m_run == -INFINITY ? 0.f : m_run;
      // P = exp2(scale * s - m) rounded to bf16, packed two per column: keys
      // half*64 .. half*64 + 63 are P columns half*32 .. half*32 + 31 of S.  The
      // row sum adds the same rounded values (two accumulators of two lanes,
      // so the adds do not form one long chain)
      uint64_t l_pair[2] = {0, 0};
      if constexpr (kCap && !kBias) {
        // tanh is monotone, so the maximum was taken on raw scores.  Below the
        // polynomials' range s P(s^2) keeps falling, past c log2e tanh(-0.4) or
        // tanh(-1); such keys' weights are below e^-20 either way when m is that far
        // above, so only the largest score is compared with the range.
        const bool none = m_run == -INFINITY;
        const bool near = none || (mt <= p.tanh_poly.near_limit && m_run + 0.379f * p.mod.cap_log2 >= 20.f * kLog2e);
        const bool wide = none || (mt <= p.tanh_poly.wide_limit && m_run + 0.761f * p.mod.cap_log2 >= 20.f * kLog2e);
        const uint64_t neg_m = pack2(-m_use, -m_use);
        if (__all_sync(0xffffffffu, near)) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            r[e] = exp2_of_pair_bf16(capped_pair(r[2 * e], r[2 * e + 1], p.tanh_poly.near, neg_m), l_pair[e % 2]);
        } else if (__all_sync(0xffffffffu, wide)) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            r[e] = exp2_of_pair_bf16(capped_pair(r[2 * e], r[2 * e + 1], p.tanh_poly.wide, neg_m), l_pair[e % 2]);
        } else {
          auto cap_all = [&](auto&& tanh_of) {
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              const float s = __uint_as_float(r[e]);
              const float z = p.mod.cap_log2 * tanh_of(s * p.mod.raw_to_x);
              r[e] = __float_as_uint(masked && s == -INFINITY ? s : z);
            }
          };
          if (p.mod.cap_log2 <= kAbsCapLog2)
            cap_all([](float x) { return tanh_by_exp_abs(x); });
          else
            cap_all([](float x) { return tanh_by_exp(x); });
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = exp2_pair_bf16(r[2 * e], r[2 * e + 1], 1.f, -m_use, l_pair[e % 2]);
        }
      } else {
        // kF16, at references whose float32 step is 2^-3 or more: the unrounded product may stand above the rounded maximum
        // by half a step, so the scores are rounded first
        if (kF16 && large) {
#pragma unroll
          for (int e = 0; e < 64; ++e) r[e] = __float_as_uint(__fmul_rn(__uint_as_float(r[e]), mul));
        }
        const float by = kF16 && large ? 1.f : mul;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          r[e] = kF16 ? exp2_pair_f16(r[2 * e], r[2 * e + 1], by, -m_use, l_pair[e % 2])
                      : exp2_pair_bf16(r[2 * e], r[2 * e + 1], mul, -m_use, l_pair[e % 2]);
      }
      tc::tmem_st32(s_addr + half * 32, r);
      float l_tile = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        l_tile += __uint_as_float(static_cast<uint32_t>(l_pair[u])) +
                  __uint_as_float(static_cast<uint32_t>(l_pair[u] >> 32));
      l_run = l_run * factor + l_tile;
      if (rescale && j > 0) {
        // O_X holds the products up to tile j-1, complete: the S_X(j) commit
        // waited on above came after them; bring this half's columns to the new
        // maximum before P_X(j) V is issued
        uint32_t o[32];
#pragma unroll
        for (int c = 0; c < kD / 64; ++c) {
          tc::tmem_ld32(o_addr + c * 32, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
          tc::tmem_st32(o_addr + c * 32, o);
        }
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[P_FULL + x]);
    }

    wait(&bars[O_FINAL + x], 0);
    tc::fence_after_sync();
    // the row sum over both halves (the exchange buffers are free: every tile's
    // maxima were read before the last P_FULL)
    *red_at(0, half) = l_run;
    named_barrier_sync(pair_id, 64);
    l_run = *red_at(0, 0) + *red_at(0, 1);
    // kInt4: where element u of eight lies among its columns
    auto column = [](int u) { return !kQ4 ? u : u < 4 ? 2 * u : 2 * u - 7; };
    // this thread's 64 outputs, 32 at a time: TMEM O (zero when the tile saw no key in this part)
    auto load_o = [&](int c, uint32_t* o) {
      if (n_x > 0) {
        tc::tmem_ld32(o_addr + c * 32, o);
        tc::tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
    };
    if (parts == 1) {
      // normalised bf16 rows staged in this tile's Q buffer (free: every MMA has
      // completed), 16-byte chunk c of row r at chunk position c ^ (r mod the
      // chunks per row) so the eight rows of a quarter-warp hit distinct banks;
      // then copied out 512 contiguous bytes (when G > 1) per warp instruction
      constexpr int kChunks = kD / 8;  // 16-byte chunks per row
      const float inv = l_run > 0.f ? (kF16 ? p.v_scale : 1.f) / l_run : 0.f;
      unsigned char* stage = sq + x * kTileQ;
#pragma unroll
      for (int c = 0; c < kD / 64; ++c) {
        uint32_t o[32];
        load_o(c, o);
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          float f[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) f[u] = __uint_as_float(o[e + column(u)]) * inv;
          const int chunk = half * (kChunks / 2) + (c * 32 + e) / 8;
          *reinterpret_cast<uint4*>(stage + row * (kD * 2) + ((chunk ^ (row & (kChunks - 1))) << 4)) =
              Chunk<__nv_bfloat16>::pack(f);
        }
      }
      named_barrier_sync(bar_id, kGroup);
#pragma unroll 4
      for (int k = 0; k < kBM * kChunks / kGroup; ++k) {
        const int rr = k * (kGroup / kChunks) + gt / kChunks;
        const int chunk = gt % kChunks;
        const int tk = tok_first + rr / G;
        if (tk < nq) {
          const uint4 v =
              *reinterpret_cast<const uint4*>(stage + rr * (kD * 2) + ((chunk ^ (rr & (kChunks - 1))) << 4));
          __nv_bfloat16* o_row = p.out + (static_cast<size_t>(q_begin + tk) * p.hq + g * G + rr % G) * kD;
          reinterpret_cast<uint4*>(o_row)[chunk] = v;
        }
      }
    } else if (tok_first < nq) {
      // Split tile: every part but the last to finish publishes O (unnormalised),
      // m and l of each row; the last waits for those records and merges.  Each
      // half handles its D / 2 columns.
      const bool row_valid = tok < nq;
      __nv_bfloat16* dst = p.out + (static_cast<size_t>(q_begin + (row_valid ? tok : 0)) * p.hq + g * G + row % G) * kD +
                           half * (kD / 2);
      const int qt = 2 * pt + x;
      const long long item = (static_cast<long long>(seq) * p.hkv + g) * p.q_tiles + qt;
      const int leader = 64 + x * kGroup;  // first thread of this tile's softmax warps
      auto record = [&](int q) {
        return reinterpret_cast<float*>(p.records + (static_cast<size_t>(item) * p.parts_max + q) * kRecordBytes);
      };
      // 16-byte chunk of this half's column d (a multiple of 4) of the thread's row:
      // the rows of a chunk are consecutive, so a warp's accesses are 512 contiguous
      // bytes
      auto record_chunk = [&](int d) { return (half * (kD / 2) + d) / 4 * kBM + row; };
      named_barrier_sync(bar_id, kGroup);
      if (threadIdx.x == leader) s_ticket[x] = atomicAdd(p.tickets + item, 1);
      named_barrier_sync(bar_id, kGroup);
      if (s_ticket[x] < parts - 1) {
        float* rec = record(part);
#pragma unroll
        for (int c = 0; c < kD / 64; ++c) {
          uint32_t o[32];
          load_o(c, o);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            reinterpret_cast<uint4*>(rec)[record_chunk(c * 32 + e)] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        if (half == 0) {
          rec[kBM * kD + row] = m_run;
          rec[kBM * kD + kBM + row] = l_run;
        }
        __threadfence();
        named_barrier_sync(bar_id, kGroup);
        if (threadIdx.x == leader) atomicAdd(p.ready + item, 1);
      } else {
        if (threadIdx.x == leader) {
          // the other parts hold their tickets, so they are resident and publish
          // soon; the wait is still bounded
          const uint64_t t0 = globaltimer_ns();
          int ok = 0;
          while (true) {
            int v;
            asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p.ready + item) : "memory");
            if (v == parts - 1) {
              ok = 1;
              break;
            }
            if (globaltimer_ns() - t0 > kSplitWaitNs) break;
            __nanosleep(100);
          }
          if (!ok) raise_error(p.err, PKV_DERR_WAIT_TIMEOUT);
          s_ticket[x] = ok ? 1 : -1;
        }
        named_barrier_sync(bar_id, kGroup);
        __threadfence();
        if (s_ticket[x] == 1) {
          // log-sum-exp merge over the parts that saw a key of this row, in part
          // order, so the result does not depend on the order they finished in
          float mq[kMaxParts], lq[kMaxParts];
          float mm = -INFINITY;
          // a part that saw no key of the row has l = 0; one with a NaN among its
          // scores must count, or the row would come out as if it had none
          constexpr float kNone = -1.f;
#pragma unroll
          for (int q = 0; q < kMaxParts; ++q) {
            mq[q] = -INFINITY;
            lq[q] = 0.f;
            if (q < parts) {
              mq[q] = q == part ? m_run : __ldcg(record(q) + kBM * kD + row);
              lq[q] = q == part ? l_run : __ldcg(record(q) + kBM * kD + kBM + row);
              if (lq[q] != 0.f) mm = fmaxf(mm, mq[q]);
            }
          }
          float total = 0.f;
#pragma unroll
          for (int q = 0; q < kMaxParts; ++q) {
            // now the part's weight, kNone where it saw no key
            mq[q] = lq[q] != 0.f ? exp2f(mq[q] - mm) : kNone;
            if (mq[q] != kNone) total += mq[q] * lq[q];
          }
          const float inv = total > 0.f ? (kF16 ? p.v_scale : 1.f) / total : 0.f;
#pragma unroll
          for (int c = 0; c < kD / 64; ++c) {
            uint32_t o[32];
            load_o(c, o);
            if (row_valid) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q0 = 0; q0 < kMaxParts; q0 += 2) {
                  if (q0 >= parts) break;
                  // two parts' loads go out before the first is used
                  float4 v[2][2];
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    if (q0 + u >= parts || q0 + u == part) continue;
                    const float4* src = reinterpret_cast<const float4*>(record(q0 + u));
                    v[u][0] = __ldcg(src + record_chunk(c * 32 + e));
                    v[u][1] = __ldcg(src + record_chunk(c * 32 + e + 4));
                  }
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    const int q = q0 + u;
                    if (q >= parts || mq[q] == kNone) continue;
                    float v8[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w, v[u][1].x, v[u][1].y, v[u][1].z, v[u][1].w};
                    if (q == part) {
#pragma unroll
                      for (int i = 0; i < 8; ++i) v8[i] = __uint_as_float(o[e + i]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] += mq[q] * v8[i];
                  }
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) f[u] *= inv;
                float elements[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) elements[u] = f[column(u)];
                reinterpret_cast<uint4*>(dst + c * 32 + e)[0] = Chunk<__nv_bfloat16>::pack(elements);
              }
            }
          }
        }
        named_barrier_sync(bar_id, kGroup);
        if (threadIdx.x == leader) {  // leave the tile's slots ready for the next call
          p.tickets[item] = 0;
          p.ready[item] = 0;
        }
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Rows per K/V copy of a paged tile: no piece crosses a block or a tile.
inline int piece_rows(const PrefillArgs& a, int tile) {
  int x = a.block_size, y = tile;
  while (y) {
    const int r = x % y;
    x = y;
    y = r;
  }
  return x;
}

template <int G, int D, Form kForm>
int launch(const PrefillArgs& a, cudaStream_t stream) {
  constexpr bool kFp8 = kForm == kE4m3;
  constexpr bool kQ4 = kForm == kInt4;
  constexpr int TQ = kBM / G;
  constexpr int kD = D;
  alignas(64) CUtensorMap tm_q, tm_k, tm_v;
  if (encode_bf16_3d(&tm_q, a.q, kD, a.hq, a.total_q, 64, G, TQ) != PKV_OK) return PKV_ECUDA;
  const bool paged = a.block_tables != nullptr;
  const int piece = paged ? piece_rows(a, kFp8 && D == 64 ? kQuarter : kBN) : kBN;
  const void* kb = paged ? a.k_cache : a.k;
  const void* vb = paged ? a.v_cache : a.v;
  const uint64_t rows = paged ? static_cast<uint64_t>(a.num_blocks) * a.block_size : a.total_k;
  if constexpr (kQ4) {
    tm_k = tm_v = tm_q;  // not used
  } else if constexpr (kFp8) {
    if (encode_u8_3d(&tm_k, kb, kD, a.hkv, rows, piece) != PKV_OK) return PKV_ECUDA;
    if (encode_u8_3d(&tm_v, vb, kD, a.hkv, rows, piece) != PKV_OK) return PKV_ECUDA;
  } else {
    if (encode_bf16_3d(&tm_k, kb, kD, a.hkv, rows, 64, 1, piece) != PKV_OK) return PKV_ECUDA;
    if (encode_bf16_3d(&tm_v, vb, kD, a.hkv, rows, 64, 1, piece) != PKV_OK) return PKV_ECUDA;
  }
  TcParams p{};
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.block_tables = a.block_tables;
  p.err = a.err;
  p.total_q = a.total_q;
  p.total_k = a.total_k;
  p.max_seqlen_q = a.max_seqlen_q;
  p.max_blocks = a.max_blocks;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.block_size = a.block_size;
  p.num_blocks = a.num_blocks;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.causal = a.causal;
  p.paged = paged ? 1 : 0;
  p.mod = a.mod;
  if constexpr (kForm == kCapped || kForm == kCappedBiased)
    p.tanh_poly = make_tanh_poly(a.mod.cap_log2, a.mod.raw_to_x);
  p.bias_mul = kForm == kBiased ? 1.f / a.scale : kLog2e;
  if constexpr (quantized(kForm)) {
    constexpr float kUp = kQ4 ? kQ4Unit : 1.f;
    p.scale_log2 = split_scale(a.scale, a.k_scale * kUp, &p.scale_exp);
    p.v_scale = a.v_scale * kUp;
    p.k_codes = static_cast<const unsigned char*>(a.k_cache);
    p.v_codes = static_cast<const unsigned char*>(a.v_cache);
  }
  if constexpr (kQ4) {
    // m = ceil(2^(31 + s) / d) with d <= 2^s: key m is off by less than 2^s key < 2^(31 + s)
    int s = 0;
    while ((1ll << s) < a.block_size) ++s;
    p.block_shift = 31 + s;
    p.block_mul = static_cast<uint32_t>(((1ull << p.block_shift) + a.block_size - 1) / a.block_size);
  }
  p.piece_rows = piece;
  const int pairs = (a.max_seqlen_q + 2 * TQ - 1) / (2 * TQ);
  p.q_tiles = 2 * pairs;
  p.parts_max = 1;
  DeviceInfo info;
  if (device_info(&info) != PKV_OK) return PKV_ECUDA;
  const size_t ws_need = prefill_tc_workspace_bytes(a.batch, a.hkv, G, D, a.max_seqlen_q);
  if (a.workspace && ws_need > 0 && a.workspace_bytes >= ws_need) {
    const long long items = static_cast<long long>(a.batch) * a.hkv * p.q_tiles;
    const size_t flags = prefill_tc_flag_bytes(items);
    unsigned char* ws = static_cast<unsigned char*>(a.workspace);
    p.parts_max = prefill_tc_parts(a.batch, a.hkv, G, a.max_seqlen_q, info.sms);
    p.tickets = reinterpret_cast<int*>(ws);
    p.ready = reinterpret_cast<int*>(ws + flags);
    p.records = ws + 2 * flags;
  }
  auto kernel = prefill_tc_kernel<G, D, kForm>;
  constexpr uint32_t kSmemBytes = Geo<D>::launch_smem(kForm);
  static std::atomic<uint64_t> smem_allowed{0};
  if (allow_smem(kernel, kSmemBytes, smem_allowed) != cudaSuccess) return PKV_ECUDA;
  dim3 grid(a.batch * a.hkv, pairs * p.parts_max);
  return launch_pdl(kernel, grid, dim3(threads(kForm)), kSmemBytes, stream, tm_q, tm_k, tm_v, p) == cudaSuccess ? PKV_OK
                                                                                                  : PKV_ECUDA;
}

template <int D, Form kForm>
int launch_d(const PrefillArgs& a, cudaStream_t stream) {
  switch (a.group) {
    case 1: return launch<1, D, kForm>(a, stream);
    case 2: return launch<2, D, kForm>(a, stream);
    case 4: return launch<4, D, kForm>(a, stream);
    default: return launch<8, D, kForm>(a, stream);
  }
}

template <Form kForm>
int launch_form(const PrefillArgs& a, cudaStream_t stream) {
  return a.head_dim == 64 ? launch_d<64, kForm>(a, stream) : launch_d<128, kForm>(a, stream);
}

}  // namespace
