// kv_rope_store: one step's q and k rotated by position, k and v stored in the
// cache ("3.6 ModelRunner, CUDA Graph, and benchmarks", section 2: the slot rule
// of kv_store; the rotation is the one the model's attention layer applies just
// before), into a cache of the rows' own type, of E4M3 codes or of 4 bits; the
// 4-bit store without rotation, and kv_load_q4, which reads 4-bit rows back.
//
// With c and s the cosines and sines of the token's position, a pair (a, b) of a
// head's first rot_dim elements becomes (a c - b s, b c + a s), rounded to
// float32, then to the rows' type, and what a quantized cache stores is that
// rounded value: the call stores bit for bit what rotating first and storing
// then would.
//
// Bound: HBM for caches of the rows' own type; q, k and v are read once, q_out and
// the cache rows written once.  Quantizing calls of many tokens are bound by latency:
// 128 registers leave 16 warps to an SM, whose issue slots are 46 % busy (8,060 tokens of
// 16 + 8 heads of 128 into 4 bits, 39 us; their bytes are 16).
#include <algorithm>
#include <cmath>

#include "q4.cuh"

namespace {

using pkv::Chunk;
using pkv::fma2;
using pkv::mul2;
using pkv::pair;
using pkv::split;

enum Format { kSame, kE4m3, kQ4 };

struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements from a token to the next
  void* q_out;
  unsigned char* k_cache;
  unsigned char* v_cache;
  const int32_t* positions;
  const float* cos_sin;
  const int32_t* slots;
  unsigned int* err;
  int num_tokens;
  int hq, hkv, head_dim, rot_dim;
  int max_position;
  int interleaved;
  int64_t num_slots;
  int row_bytes;  // of a token in the cache
  float k_scale, v_scale;
};

// Eight consecutive elements of a row.
template <typename T>
struct Run {
  static constexpr int kWords = 8 / Chunk<T>::N;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) Chunk<T>::unpack(w[i], f + i * Chunk<T>::N);
  }
  __device__ __forceinline__ void pack(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = Chunk<T>::pack(f + i * Chunk<T>::N);
  }
};

// a c - b s (kMinus) or a c + b s, correct to 2^-46 of its terms before the one
// rounding: both products are taken with their errors, and their sum with its
// own.  A key next to the border of two codes, or of two bf16 values, then falls
// on its side whatever the order of operations of whoever checks it.
template <bool kMinus>
__device__ __forceinline__ float turn(float a, float b, float c, float s) {
  const float bs = kMinus ? -b : b;
  const float p = __fmul_rn(a, c), q = __fmul_rn(bs, s);
  const float ep = __fmaf_rn(a, c, -p), eq = __fmaf_rn(bs, s, -q);
  const float h = __fadd_rn(p, q);
  const float t = __fadd_rn(h, -p);
  const float eh = __fadd_rn(__fadd_rn(p, -__fadd_rn(h, -t)), __fadd_rn(q, -t));
  const float r = __fadd_rn(h, __fadd_rn(eh, __fadd_rn(ep, eq)));
  return fabsf(h) <= 3.402823466e38f ? r : h;  // infinities and NaN have no error term
}

// Two floats rounded to bf16; `near` keeps the least distance (in 16-bit halves) from four
// units in the last place below the middle of two bf16 numbers.
__device__ __forceinline__ uint32_t round_pair(uint64_t y, uint32_t& near) {
  float a, b;
  split(y, a, b);
  near = __viaddmin_u16x2(pkv::prmt(__float_as_uint(a), __float_as_uint(b), 0x5410u), 0x80048004u, near);
  return pkv::pack_bf16x2(a, b);
}

// Eight pairs (a, b), two to a word, turned by (c, s) and rounded to bf16.
// kAcross: the result pairs stay as they are, else (a, b) become neighbours.
// Kahan's a c + b t = fma(a, c, fl(b t)) + (b t - fl(b t)) is off by at most 1.5
// units in the last place, which bf16's rounding forgets but for values next to
// the middle of two bf16 numbers: those (one in 2^13), and NaN, which an infinite
// product gives, are taken again with turn().  Four instructions for two elements
// where turn() takes 17 for one.
template <bool kAcross>
__device__ __forceinline__ void turn_pairs(const uint64_t (&a)[4], const uint64_t (&b)[4], const float (&c)[8],
                                           const float (&s)[8], uint32_t (&x)[4], uint32_t (&y)[4]) {
  const uint64_t minus = pair(-1.f, -1.f);
  uint32_t near = 0xffffffffu;
  uint64_t nan = 0ull;
  uint32_t ra[4], rb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t c2 = pair(c[2 * i], c[2 * i + 1]), s2 = pair(s[2 * i], s[2 * i + 1]);
    const uint64_t n2 = pair(-s[2 * i], -s[2 * i + 1]);
    const uint64_t wa = mul2(b[i], n2), wb = mul2(a[i], s2);
    const uint64_t ya = fma2(fma2(b[i], s2, wa), minus, fma2(a[i], c2, wa));
    const uint64_t yb = fma2(fma2(a[i], n2, wb), minus, fma2(b[i], c2, wb));
    nan = fma2(ya, 0ull, fma2(yb, 0ull, nan));
    ra[i] = round_pair(ya, near);
    rb[i] = round_pair(yb, near);
  }
  float n0, n1;
  split(nan, n0, n1);
  if ((near & 0xffffu) <= 8u || near <= 0x8ffffu || !(n0 + n1 == 0.f)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a2[2], b2[2], ya[2], yb[2];
      split(a[i], a2[0], a2[1]);
      split(b[i], b2[0], b2[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ya[e] = turn<true>(a2[e], b2[e], c[2 * i + e], s[2 * i + e]);
        yb[e] = turn<false>(b2[e], a2[e], c[2 * i + e], s[2 * i + e]);
      }
      ra[i] = pkv::pack_bf16x2(ya[0], ya[1]);
      rb[i] = pkv::pack_bf16x2(yb[0], yb[1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kAcross) {
      x[i] = ra[i];
      y[i] = rb[i];
    } else {
      uint32_t(&out)[4] = i < 2 ? x : y;
      out[2 * (i & 1)] = pkv::prmt(ra[i], rb[i], 0x5410u);
      out[2 * (i & 1) + 1] = pkv::prmt(ra[i], rb[i], 0x7632u);
    }
  }
}

__device__ __forceinline__ uint64_t low_pair(uint32_t x, uint32_t y) {
  return pair(__uint_as_float(x << 16), __uint_as_float(y << 16));
}
__device__ __forceinline__ uint64_t high_pair(uint32_t x, uint32_t y) {
  return pair(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u));
}

// Turns two runs: element i of the one with element i of the other by (c[i], s[i]),
// or, interleaved, the neighbours of each run, four pairs by the first four angles
// and four by the last.
__device__ __forceinline__ void rotate(Run<__nv_bfloat16>& r0, Run<__nv_bfloat16>& r1, const float (&c)[8],
                                       const float (&s)[8], bool interleaved) {
  uint32_t x[4] = {r0.w[0].x, r0.w[0].y, r0.w[0].z, r0.w[0].w}, y[4] = {r1.w[0].x, r1.w[0].y, r1.w[0].z, r1.w[0].w};
  uint64_t a[4], b[4];
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = pair(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u));
      b[i] = pair(__uint_as_float(y[i] << 16), __uint_as_float(y[i] & 0xffff0000u));
    }
    turn_pairs<true>(a, b, c, s, x, y);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = low_pair(x[2 * i], x[2 * i + 1]);
      b[i] = high_pair(x[2 * i], x[2 * i + 1]);
      a[2 + i] = low_pair(y[2 * i], y[2 * i + 1]);
      b[2 + i] = high_pair(y[2 * i], y[2 * i + 1]);
    }
    turn_pairs<false>(a, b, c, s, x, y);
  }
  r0.w[0] = make_uint4(x[0], x[1], x[2], x[3]);
  r1.w[0] = make_uint4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ void rotate(Run<float>& r0, Run<float>& r1, const float (&c)[8], const float (&s)[8],
                                       bool interleaved) {
  float x0[8], x1[8];
  r0.unpack(x0);
  r1.unpack(x1);
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y0 = turn<true>(x0[i], x1[i], c[i], s[i]);
      x1[i] = turn<false>(x1[i], x0[i], c[i], s[i]);
      x0[i] = y0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y0 = turn<true>(x0[2 * i], x0[2 * i + 1], c[i], s[i]);
      x0[2 * i + 1] = turn<false>(x0[2 * i + 1], x0[2 * i], c[i], s[i]);
      x0[2 * i] = y0;
      const float y1 = turn<true>(x1[2 * i], x1[2 * i + 1], c[4 + i], s[4 + i]);
      x1[2 * i + 1] = turn<false>(x1[2 * i + 1], x1[2 * i], c[4 + i], s[4 + i]);
      x1[2 * i] = y1;
    }
  }
  r0.pack(x0);
  r1.pack(x1);
}

// Writes eight elements at `dim` of a head's row in the cache.  Lanes 2i and
// 2i + 1 hold the two halves of a group of 16 (kQ4: both must be here).
template <typename T, Format kFormat>
__device__ __forceinline__ void store_cache(const RopeArgs& a, unsigned char* row, int head, int dim, const Run<T>& run,
                                            float scale, bool valid) {
  if constexpr (kFormat == kSame) {
    if (valid) run.store(reinterpret_cast<T*>(row) + head * a.head_dim + dim);
    return;
  }
  float x[8];
  run.unpack(x);
  if constexpr (kFormat == kE4m3) {
    const uint2 codes = pkv::e4m3_codes8(x, scale);
    if (valid) *reinterpret_cast<uint2*>(row + head * a.head_dim + dim) = codes;
  } else {
    // (the group's largest magnitude, on bf16 pairs)
    uint32_t top2 = 0u;
    const uint32_t words[4] = {run.w[0].x, run.w[0].y, run.w[0].z, run.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top2) : "r"(words[i] & 0x7fff7fffu));
    float top = pkv::max_keep_nan(__uint_as_float(top2 << 16), __uint_as_float(top2 & 0xffff0000u));
    top = pkv::max_keep_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const uint32_t code = pkv::q4_scale_code(top, scale);
    const uint32_t w = pkv::q4_codes8(x, code, scale);
    if (valid) {
      *reinterpret_cast<uint32_t*>(row + (head * a.head_dim + dim) / 2) = w;
      if ((dim & 8) == 0)
        row[pkv::q4_scale_offset(a.hkv, a.head_dim) + (head * a.head_dim + dim) / 16] = static_cast<unsigned char>(code);
    }
  }
}

// What a thread takes of a head: two runs of eight elements.  Of the rotated part
// the runs that pair with each other (element i of the first half and of the
// second; with neighbouring pairs the same runs, each by itself), of the rest and
// of V the runs half the length apart.  Runs 2i and 2i + 1 of a head, the halves of
// a group of 16, lie in neighbouring lanes.
template <typename T, Format kFormat, bool kRope>
struct Lane {
  const RopeArgs& a;
  bool turned;
  int j, v0, v1, d0, d1;
  float c[8], s[8];

  __device__ __forceinline__ Lane(const RopeArgs& args, int unit) : a(args), j(unit) {
    turned = kRope && j < a.rot_dim / 16;
    v0 = j * 8;
    v1 = a.head_dim / 2 + j * 8;
    d0 = v0;
    d1 = v1;
    if (turned) {
      d1 = a.rot_dim / 2 + j * 8;
    } else if (kRope) {
      d0 = a.rot_dim / 2 + j * 8;
      d1 = d0 + (a.head_dim - a.rot_dim) / 2;
    }
  }
  __device__ __forceinline__ void angles(const float* row) {
    const int half = a.rot_dim / 2;
    // (interleaved: pairs 4j .. 4j + 3 in the first run, rot_dim / 4 further on in the second)
    const int at = a.interleaved ? j * 4 : j * 8, next = a.interleaved ? half / 2 : 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 cv = *reinterpret_cast<const float4*>(row + at + i * next);
      const float4 sv = *reinterpret_cast<const float4*>(row + half + at + i * next);
      c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
      s[4 * i] = sv.x, s[4 * i + 1] = sv.y, s[4 * i + 2] = sv.z, s[4 * i + 3] = sv.w;
    }
  }
  // The runs of head h (of q, k, v in turn), zeros when it is not `here`.
  __device__ __forceinline__ void load(int h, const T* src, bool here, Run<T>& r0, Run<T>& r1) const {
    const bool is_v = h >= a.hq + a.hkv;
    r0.clear();
    r1.clear();
    if (here) {
      r0.load(src + (is_v ? v0 : d0));
      r1.load(src + (is_v ? v1 : d1));
    }
  }
  // Turns and writes them: `kept`, the token has a position (and the lane a head), `stored`, a
  // slot too.  Every lane of the warp calls it.
  __device__ __forceinline__ void finish(int h, int token, int64_t slot, bool kept, bool stored, Run<T>& r0,
                                         Run<T>& r1) const {
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
    const int e0 = is_v ? v0 : d0, e1 = is_v ? v1 : d1;
    if (kept) {
      if (turned && !is_v) rotate(r0, r1, c, s, a.interleaved);
      if (is_q) {
        T* dst = static_cast<T*>(a.q_out) + (static_cast<int64_t>(token) * a.hq + h) * a.head_dim;
        r0.store(dst + e0);
        r1.store(dst + e1);
      }
    }
    if (!__any_sync(0xffffffffu, stored && !is_q)) return;
    const bool write = stored && !is_q;
    unsigned char* row = (is_v ? a.v_cache : a.k_cache) + (write ? slot * a.row_bytes : 0);
    const int in_cache = is_v ? h - a.hq - a.hkv : h - a.hq;
    const float scale = is_v ? a.v_scale : a.k_scale;
    store_cache<T, kFormat>(a, row, in_cache, e0, r0, scale, write);
    store_cache<T, kFormat>(a, row, in_cache, e1, r1, scale, write);
  }
};

// A token's heads go round `lanes` threads of a block, kBatch at a time, whose loads go out together.
template <typename T, Format kFormat, bool kRope, int kBatch>
__global__ void __launch_bounds__(256) kv_rope_store_kernel(const RopeArgs a, int lanes, int tokens_per_block) {
  pkv::pdl_enter();
  const int per_head = a.head_dim / 16;
  const int per_token = lanes * per_head;
  const int in_block = threadIdx.x / per_token;
  const int w = threadIdx.x - in_block * per_token;
  const int token = blockIdx.x * tokens_per_block + in_block;
  const bool here = in_block < tokens_per_block && token < a.num_tokens;
  Lane<T, kFormat, kRope> lane(a, w % per_head);
  const int64_t slot = here ? __ldg(a.slots + token) : -1;
  const int position = kRope && here ? __ldg(a.positions + token) : 0;
  const int heads = a.hq + 2 * a.hkv;
  bool kept = here, stored = false;
  for (int h0 = w / per_head; h0 - w / per_head < heads; h0 += kBatch * lanes) {
    Run<T> r0[kBatch], r1[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * lanes;
      const T* src = h < a.hq           ? static_cast<const T*>(a.q) + token * a.q_stride + h * a.head_dim
                     : h < a.hq + a.hkv ? static_cast<const T*>(a.k) + token * a.k_stride + (h - a.hq) * a.head_dim
                                        : static_cast<const T*>(a.v) + token * a.v_stride +
                                              (h - a.hq - a.hkv) * a.head_dim;
      lane.load(h, src, here && h < heads, r0[i], r1[i]);
    }
    if (h0 < lanes) {  // (after the first loads)
      stored = here && slot >= 0 && slot < a.num_slots;
      if (here && !stored && slot != -1 && w == 0) pkv::raise_error(a.err, PKV_DERR_SLOT_RANGE);
      if (kRope && here && (position < 0 || position >= a.max_position)) {
        if (w == 0) pkv::raise_error(a.err, PKV_DERR_POSITION_RANGE);
        kept = stored = false;
      }
      if (lane.turned && kept) lane.angles(a.cos_sin + static_cast<int64_t>(position) * a.rot_dim);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * lanes;
      lane.finish(h, token, slot, kept && h < heads, stored && h < heads, r0[i], r1[i]);
    }
  }
}

// Many large tokens into a cache of their own type: one block per SM, each warp
// streams pieces of tokens (consecutive heads, about 4 KB of them) through a ring of
// its own that bulk copies fill, the row of angles with them, so that what is in
// flight does not depend on registers.  65,536 tokens of 16 + 8 heads of 128 in bf16:
// 184 us, 87 % of a copy's rate, where four heads to a thread take 225.  It is for
// tokens that fill a piece (32,768 of 8 + 1 heads of 64: 35 us, 23 with four heads to a
// thread).  Quantized caches gain nothing from it as it is: it has the same 16 warps per
// SM as the other (32,768 tokens of 16 + 8 heads, E4M3: 119 us against 123, 4 bits: 139
// against 136).
constexpr int kStreamWarps = 16;
constexpr int kStreamStages = 3;
constexpr int kStageBytes = 4608;  // 16 heads of 128 bf16 and their angles; at most, a head and angles of 2 KB each
constexpr int kStreamSmem = kStreamWarps * kStreamStages * (kStageBytes + 8);

template <typename T>
__global__ void __launch_bounds__(kStreamWarps * 32, 1) kv_rope_stream_kernel(const RopeArgs a, int piece_heads,
                                                                              int pieces) {
  pkv::pdl_enter();
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x / 32, tid = threadIdx.x % 32;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem) + warp * kStreamStages;
  unsigned char* ring = smem + kStreamWarps * kStreamStages * 8 + warp * kStreamStages * kStageBytes;
  if (tid == 0) {
    for (int i = 0; i < kStreamStages; ++i) pkv::mbar_init(&full[i], 1);
    pkv::fence_mbar_init();
  }
  __syncwarp();
  const int heads = a.hq + 2 * a.hkv;
  const int head_bytes = a.head_dim * static_cast<int>(sizeof(T));
  const int angles_at = piece_heads * head_bytes;
  const int per_head = a.head_dim / 16, side = 32 / per_head;  // heads side by side
  Lane<T, kSame, true> lane(a, tid % per_head);
  const int mine = tid / per_head < side ? tid / per_head : heads;
  const int64_t items = static_cast<int64_t>(a.num_tokens) * pieces;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kStreamWarps;
  const uint64_t policy = pkv::l2_evict_first_policy();

  struct Item {
    int token, piece, position;
    int64_t slot;
  };
  auto look_up = [&](int64_t item) {
    Item it{-1, 0, 0, -1};
    if (item < items) {
      it.token = static_cast<int>(item / pieces);
      it.piece = static_cast<int>(item - static_cast<int64_t>(it.token) * pieces);
      it.slot = __ldg(a.slots + it.token);
      it.position = __ldg(a.positions + it.token);
    }
    return it;
  };
  auto placed = [&](const Item& it) { return it.position >= 0 && it.position < a.max_position; };
  auto copy = [&](const Item& it, int st) {
    if (tid != 0 || it.token < 0) return;
    unsigned char* dst = ring + st * kStageBytes;
    const int first = it.piece * piece_heads, end = min(first + piece_heads, heads);
    const bool angles = placed(it);
    pkv::mbar_expect_tx(&full[st], (end - first) * head_bytes + (angles ? a.rot_dim * 4 : 0));
    auto part = [&](const void* base, int64_t stride, int from, int count) {
      const int lo = max(first, from), hi = min(end, from + count);
      if (lo < hi)
        pkv::bulk_g2s(dst + (lo - first) * head_bytes,
                      static_cast<const T*>(base) + it.token * stride + (lo - from) * a.head_dim, (hi - lo) * head_bytes,
                      &full[st], policy);
    };
    part(a.q, a.q_stride, 0, a.hq);
    part(a.k, a.k_stride, a.hq, a.hkv);
    part(a.v, a.v_stride, a.hq + a.hkv, a.hkv);
    if (angles)
      pkv::bulk_g2s(dst + angles_at, a.cos_sin + static_cast<int64_t>(it.position) * a.rot_dim, a.rot_dim * 4, &full[st],
                    pkv::l2_normal_policy());
    pkv::mbar_arrive(&full[st]);
  };
  int64_t next = static_cast<int64_t>(blockIdx.x) * kStreamWarps + warp;
  Item queue[kStreamStages];
#pragma unroll
  for (int i = 0; i < kStreamStages; ++i, next += step) {
    queue[i] = look_up(next);
    copy(queue[i], i);
  }
  int st = 0;
  uint32_t parity = 0;
  while (queue[0].token >= 0) {
    const Item coming = look_up(next);
    next += step;
    const Item it = queue[0];
    if (!__all_sync(0xffffffffu, pkv::mbar_wait(&full[st], parity))) {  // (the lanes leave together)
      if (tid == 0) pkv::raise_error(a.err, PKV_DERR_WAIT_TIMEOUT);
      // the block must not end with copies on their way into its shared memory
#pragma unroll
      for (int i = 0; i < kStreamStages; ++i)
        if (queue[i].token >= 0)
          pkv::mbar_wait(&full[(st + i) % kStreamStages], st + i >= kStreamStages ? parity ^ 1u : parity);
      return;
    }
    const unsigned char* src = ring + st * kStageBytes;
    const bool kept = placed(it);
    const bool slot_ok = it.slot >= 0 && it.slot < a.num_slots;
    if (tid == 0 && it.piece == 0) {
      if (!slot_ok && it.slot != -1) pkv::raise_error(a.err, PKV_DERR_SLOT_RANGE);
      if (!kept) pkv::raise_error(a.err, PKV_DERR_POSITION_RANGE);
    }
    if (lane.turned && kept) lane.angles(reinterpret_cast<const float*>(src + angles_at));
    const int first = it.piece * piece_heads, count = min(piece_heads, heads - first);
#pragma unroll 2
    for (int h0 = 0; h0 < count; h0 += side) {
      const bool here = kept && h0 + mine < count;
      Run<T> r0, r1;
      lane.load(first + h0 + mine, reinterpret_cast<const T*>(src + (h0 + mine) * head_bytes), here, r0, r1);
      lane.finish(first + h0 + mine, it.token, it.slot, here, here && slot_ok, r0, r1);
    }
    __syncwarp();  // the stage has been read
    copy(coming, st);
#pragma unroll
    for (int i = 0; i + 1 < kStreamStages; ++i) queue[i] = queue[i + 1];
    queue[kStreamStages - 1] = coming;
    if (++st == kStreamStages) {
      st = 0;
      parity ^= 1u;
    }
  }
}

// Threads of a token's heads, and tokens of a block of 256.
struct Split {
  int lanes, tokens;
  Split(int heads, int units_per_head, int batch)
      : lanes(std::min((heads + batch - 1) / batch, 256 / units_per_head)), tokens(256 / (lanes * units_per_head)) {}
  unsigned blocks(int64_t num_tokens) const { return static_cast<unsigned>((num_tokens + tokens - 1) / tokens); }
};
// More work than one head to a thread keeps on the GPU at once.
bool many(int num_tokens, int units, int sms) { return static_cast<int64_t>(num_tokens) * units > sms * 1024ll; }

template <typename T, Format kFormat, bool kRope>
int launch_store(const RopeArgs& a, cudaStream_t stream) {
  pkv::DeviceInfo info;
  if (pkv::device_info(&info) != PKV_OK) return PKV_ECUDA;
  const int heads = a.hq + 2 * a.hkv, per_head = a.head_dim / 16;
  const bool batch = many(a.num_tokens, heads * per_head, info.sms);
  if constexpr (kFormat == kSame) {
    const int head_bytes = a.head_dim * static_cast<int>(sizeof(T));
    const int piece_heads = (kStageBytes - a.rot_dim * 4) / head_bytes;
    if (batch && heads >= piece_heads) {
      static std::atomic<uint64_t> smem_allowed{0};
      if (pkv::allow_smem(kv_rope_stream_kernel<T>, kStreamSmem, smem_allowed) != cudaSuccess) return PKV_ECUDA;
      return pkv::launch_pdl(kv_rope_stream_kernel<T>, dim3(info.sms), dim3(kStreamWarps * 32), kStreamSmem, stream, a,
                             piece_heads, (heads + piece_heads - 1) / piece_heads) == cudaSuccess
                 ? PKV_OK
                 : PKV_ECUDA;
    }
  }
  const Split split(heads, per_head, batch ? 4 : 1);
  auto kernel = batch ? kv_rope_store_kernel<T, kFormat, kRope, 4> : kv_rope_store_kernel<T, kFormat, kRope, 1>;
  return pkv::launch_pdl(kernel, dim3(split.blocks(a.num_tokens)), dim3(256), 0, stream, a, split.lanes, split.tokens) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

struct LoadArgs {
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  const unsigned char* k_cache;
  const unsigned char* v_cache;
  const int32_t* slots;
  unsigned int* err;
  int num_tokens, hkv, head_dim, row_bytes;
  int64_t num_slots;
  float k_scale, v_scale;
};

// A thread takes eight elements of kBatch of a token's 2 hkv heads: a word of codes
// and the group's scale byte become 16 bytes of bf16.  (code - 8) * scale is exact
// in f16; the tensor's scale is applied in float32, one rounding, then bf16's.
template <int kBatch>
__global__ void __launch_bounds__(256) kv_load_q4_kernel(const LoadArgs a, int lanes, int tokens_per_block) {
  pkv::pdl_enter();
  const int per_head = a.head_dim / 8;
  const int per_token = lanes * per_head;
  const int in_block = threadIdx.x / per_token;
  const int w = threadIdx.x - in_block * per_token;
  const int lane = w / per_head, j = w - lane * per_head;
  const int token = blockIdx.x * tokens_per_block + in_block;
  if (in_block >= tokens_per_block || token >= a.num_tokens) return;
  const int64_t slot = __ldg(a.slots + token);
  const bool valid = slot >= 0 && slot < a.num_slots;
  if (!valid && slot != -1 && w == 0) pkv::raise_error(a.err, PKV_DERR_SLOT_RANGE);
  const int64_t row = valid ? slot * a.row_bytes : 0;
  const int scales = pkv::q4_scale_offset(a.hkv, a.head_dim);
  for (int h0 = 0; h0 < 2 * a.hkv; h0 += kBatch * lanes) {
    uint32_t codes[kBatch], scale[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * lanes + lane;
      const int head = h >= a.hkv ? h - a.hkv : h;
      codes[i] = scale[i] = 0u;  // (a scale of 0: zeros)
      if (valid && h < 2 * a.hkv) {
        const unsigned char* src = (h >= a.hkv ? a.v_cache : a.k_cache) + row;
        codes[i] = __ldg(reinterpret_cast<const uint32_t*>(src) + head * per_head + j);
        scale[i] = __ldg(src + scales + (head * per_head + j) / 2);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * lanes + lane;
      if (h >= 2 * a.hkv) break;
      const bool is_v = h >= a.hkv;
      const int head = is_v ? h - a.hkv : h;
      uint32_t f[4];  // elements (0, 4), (1, 5), (2, 6), (3, 7), over 64
      pkv::widen_q4(codes[i], pkv::Q4Scale(pkv::prmt(pkv::e4m3x2_to_f16x2(scale[i]), 0, 0x1010u)), f);
      const float tensor = is_v ? a.v_scale : a.k_scale;
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t whole = pkv::hmul2(f[e], 0x54005400u);
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&whole));
        x[e] = __fmul_rn(y.x, tensor);
        x[e + 4] = __fmul_rn(y.y, tensor);
      }
      __nv_bfloat16* dst = (is_v ? a.v : a.k) + (static_cast<int64_t>(token) * a.hkv + head) * a.head_dim;
      reinterpret_cast<uint4*>(dst)[j] = Chunk<__nv_bfloat16>::pack(x);
    }
  }
}

bool scale_ok(float s) { return s > 0.f && !std::isinf(s); }

// What both stores check; PKV_OK when a launch may follow, 1 when there is nothing to do.
int check_store(const RopeArgs& a, int num_blocks, int block_size, int format, int elt) {
  if (a.num_tokens < 0 || num_blocks < 0 || block_size <= 0 || a.hkv <= 0 || a.hq < 0 || a.head_dim <= 0)
    return PKV_EINVAL;
  if (format == PKV_CACHE_E4M3 || format == PKV_CACHE_Q4)
    if (!scale_ok(a.k_scale) || !scale_ok(a.v_scale)) return PKV_EINVAL;
  if (format == PKV_CACHE_Q4 && !pkv::q4_head_dim(a.head_dim)) return PKV_EUNSUPPORTED;
  if (a.head_dim % 32 != 0 || a.head_dim > 512 || a.hq > 1024 || a.hkv > 1024) return PKV_EUNSUPPORTED;
  if (static_cast<long long>(num_blocks) * block_size > INT32_MAX) return PKV_EINVAL;
  if (a.num_tokens == 0) return 1;
  if (!a.k || !a.v || !a.k_cache || !a.v_cache || !a.slots) return PKV_EINVAL;
  const void* pointers[] = {a.q, a.k, a.v, a.q_out, a.k_cache, a.v_cache, a.cos_sin};
  for (const void* p : pointers)
    if (!pkv::aligned16(p)) return PKV_EALIGN;
  const int64_t strides[] = {a.q_stride, a.k_stride, a.v_stride};
  const int heads[] = {a.hq, a.hkv, a.hkv};
  for (int i = 0; i < 3; ++i) {
    if (heads[i] == 0) continue;
    if (strides[i] < static_cast<int64_t>(heads[i]) * a.head_dim) return PKV_EINVAL;
    if (strides[i] * elt % 16 != 0) return PKV_EALIGN;
  }
  return PKV_OK;
}

}  // namespace

extern "C" int64_t pkv_q4_row_bytes(int32_t num_kv_heads, int32_t head_dim) {
  if (num_kv_heads <= 0 || num_kv_heads > 1024 || !pkv::q4_head_dim(head_dim)) return 0;
  return pkv::q4_row_bytes(num_kv_heads, head_dim);
}

extern "C" int pkv_kv_rope_store(void* q_out, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                 const void* v, int64_t v_stride, const int32_t* positions, const float* cos_sin,
                                 int32_t max_position, int32_t rot_dim, int32_t interleaved, void* k_cache,
                                 void* v_cache, const int32_t* slot_mapping, int32_t num_tokens, int32_t num_blocks,
                                 int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                 pkv_cache_format format, float k_scale, float v_scale, pkv_dtype dtype,
                                 pkv_stream_t stream) {
  if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_EUNSUPPORTED;
  if (format != PKV_CACHE_SAME && format != PKV_CACHE_E4M3 && format != PKV_CACHE_Q4) return PKV_EUNSUPPORTED;
  if (format != PKV_CACHE_SAME && dtype != PKV_BF16) return PKV_EUNSUPPORTED;
  if (num_q_heads <= 0 || rot_dim <= 0 || max_position < 0 || (interleaved != 0 && interleaved != 1)) return PKV_EINVAL;
  if (rot_dim > head_dim) return PKV_EINVAL;
  if (rot_dim % 32 != 0) return PKV_EUNSUPPORTED;
  const int elt = dtype == PKV_F32 ? 4 : 2;
  RopeArgs a{q, k, v, q_stride, k_stride, v_stride, q_out, static_cast<unsigned char*>(k_cache),
             static_cast<unsigned char*>(v_cache), positions, cos_sin, slot_mapping, nullptr, num_tokens, num_q_heads,
             num_kv_heads, head_dim, rot_dim, max_position, interleaved, static_cast<int64_t>(num_blocks) * block_size, 0,
             k_scale, v_scale};
  const int chk = check_store(a, num_blocks, block_size, format, elt);
  if (chk != PKV_OK) return chk > 0 ? PKV_OK : chk;
  if (!q || !q_out || !positions || !cos_sin) return PKV_EINVAL;
  // in place only row by row: with another stride a token's output would land on another's input
  if (q_out == q && q_stride != static_cast<int64_t>(num_q_heads) * head_dim) return PKV_EINVAL;
  a.row_bytes = format == PKV_CACHE_Q4 ? pkv::q4_row_bytes(num_kv_heads, head_dim)
                                       : num_kv_heads * head_dim * (format == PKV_CACHE_E4M3 ? 1 : elt);
  int st = PKV_OK;
  a.err = pkv::device_error_word(&st);
  if (st != PKV_OK) return st;
  if (dtype == PKV_F32) return launch_store<float, kSame, true>(a, stream);
  if (format == PKV_CACHE_SAME) return launch_store<__nv_bfloat16, kSame, true>(a, stream);
  if (format == PKV_CACHE_E4M3) return launch_store<__nv_bfloat16, kE4m3, true>(a, stream);
  return launch_store<__nv_bfloat16, kQ4, true>(a, stream);
}

extern "C" int pkv_kv_store_q4(const void* k, const void* v, void* k_cache, void* v_cache, const int32_t* slot_mapping,
                               int32_t num_tokens, int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                               int32_t head_dim, float k_scale, float v_scale, pkv_stream_t stream) {
  const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
  RopeArgs a{};
  a.k = k;
  a.v = v;
  a.k_stride = a.v_stride = row;
  a.k_cache = static_cast<unsigned char*>(k_cache);
  a.v_cache = static_cast<unsigned char*>(v_cache);
  a.slots = slot_mapping;
  a.num_tokens = num_tokens;
  a.hkv = num_kv_heads;
  a.head_dim = head_dim;
  a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const int chk = check_store(a, num_blocks, block_size, PKV_CACHE_Q4, 2);
  if (chk != PKV_OK) return chk > 0 ? PKV_OK : chk;
  a.row_bytes = pkv::q4_row_bytes(num_kv_heads, head_dim);
  int st = PKV_OK;
  a.err = pkv::device_error_word(&st);
  if (st != PKV_OK) return st;
  return launch_store<__nv_bfloat16, kQ4, false>(a, stream);
}

extern "C" int pkv_kv_load_q4(void* k, void* v, const void* k_cache, const void* v_cache, const int32_t* slot_mapping,
                              int32_t num_tokens, int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                              int32_t head_dim, float k_scale, float v_scale, pkv_stream_t stream) {
  if (num_tokens < 0 || num_blocks < 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0) return PKV_EINVAL;
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return PKV_EINVAL;
  if (!pkv::q4_head_dim(head_dim) || num_kv_heads > 1024) return PKV_EUNSUPPORTED;
  if (static_cast<long long>(num_blocks) * block_size > INT32_MAX) return PKV_EINVAL;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !k_cache || !v_cache || !slot_mapping) return PKV_EINVAL;
  if (!pkv::aligned16(k) || !pkv::aligned16(v) || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache))
    return PKV_EALIGN;
  int st = PKV_OK;
  unsigned int* err = pkv::device_error_word(&st);
  if (st != PKV_OK) return st;
  pkv::DeviceInfo info;
  if (pkv::device_info(&info) != PKV_OK) return PKV_ECUDA;
  const LoadArgs a{static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), static_cast<const unsigned char*>(k_cache),
                   static_cast<const unsigned char*>(v_cache), slot_mapping, err, num_tokens, num_kv_heads, head_dim,
                   pkv::q4_row_bytes(num_kv_heads, head_dim), static_cast<int64_t>(num_blocks) * block_size, k_scale, v_scale};
  const int per_head = head_dim / 8;
  const bool batch = many(num_tokens, 2 * num_kv_heads * per_head, info.sms);
  const Split split(2 * num_kv_heads, per_head, batch ? 4 : 1);
  return pkv::launch_pdl(batch ? kv_load_q4_kernel<4> : kv_load_q4_kernel<1>, dim3(split.blocks(num_tokens)), dim3(256), 0,
                         stream, a, split.lanes, split.tokens) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}
