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
// Bound: HBM.  q, k and v are read once, q_out and the cache rows written once;
// the table rows are shared by a token's heads in L1.
#include <algorithm>
#include <cmath>

#include "q4.cuh"

namespace {

using pkv::Chunk;

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

// Eight consecutive elements as floats.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  const uint4* src = reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < 8 / Chunk<T>::N; ++i) Chunk<T>::unpack(src[i], f + i * Chunk<T>::N);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  uint4* dst = reinterpret_cast<uint4*>(p);
#pragma unroll
  for (int i = 0; i < 8 / Chunk<T>::N; ++i) dst[i] = Chunk<T>::pack(f + i * Chunk<T>::N);
}

// a c - b s (kMinus) or a c + b s, correct to 2^-46 of its terms before the one
// rounding: both products are taken with their errors, and their sum with its
// own.  A quantized key next to the border of two codes then falls on its side
// whatever the order of operations of whoever checks it; the store has the time
// (it waits for memory).
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

template <typename T>
__device__ __forceinline__ float rounded(float x);
template <>
__device__ __forceinline__ float rounded<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ float rounded<__nv_bfloat16>(float x) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

// Writes eight elements at `dim` of a head's row in the cache.  Lanes 2i and
// 2i + 1 hold the two halves of a group of 16 (kQ4: both must be here).
template <typename T, Format kFormat>
__device__ __forceinline__ void store_cache(const RopeArgs& a, unsigned char* cache, int64_t slot, int head, int dim,
                                            const float (&x)[8], float scale, bool valid) {
  unsigned char* row = cache + slot * a.row_bytes;
  if constexpr (kFormat == kSame) {
    if (valid) store8(reinterpret_cast<T*>(row) + head * a.head_dim + dim, x);
  } else if constexpr (kFormat == kE4m3) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t code[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) code[j] = pkv::to_e4m3(__fdiv_rn(x[4 * i + j], scale));
      w[i] = code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24;
    }
    if (valid) *reinterpret_cast<uint2*>(row + head * a.head_dim + dim) = make_uint2(w[0], w[1]);
  } else {
    float top = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) top = pkv::max_keep_nan(top, fabsf(x[i]));
    top = pkv::max_keep_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const uint32_t code = pkv::to_e4m3(__fdiv_rn(top, __fmul_rn(7.f, scale)));
    const uint32_t w = pkv::q4_codes8(x, code, scale);
    if (valid) {
      *reinterpret_cast<uint32_t*>(row + (head * a.head_dim + dim) / 2) = w;
      if ((dim & 8) == 0)
        row[pkv::q4_scale_offset(a.hkv, a.head_dim) + (head * a.head_dim + dim) / 16] = static_cast<unsigned char>(code);
    }
  }
}

// A thread takes two runs of eight elements of one head: of the rotated part the
// runs that pair with each other (element i of the first half and of the second;
// with neighbouring pairs the same runs, each by itself), of the rest and of V the
// runs half the length apart.  Runs 2i and 2i + 1 of a head, the halves of a
// group of 16, lie in neighbouring lanes.
template <typename T, Format kFormat, bool kRope>
__global__ void __launch_bounds__(256) kv_rope_store_kernel(const RopeArgs a, int tokens_per_block) {
  pkv::pdl_enter();
  const int per_head = a.head_dim / 16;
  const int per_token = (a.hq + 2 * a.hkv) * per_head;
  const int total = tokens_per_block * per_token;
  const int turned = a.rot_dim / 16;
  for (int u0 = threadIdx.x & ~31; u0 < total; u0 += blockDim.x) {
    const int u = u0 + static_cast<int>(threadIdx.x & 31);
    const int in_block = u / per_token;
    const int token = blockIdx.x * tokens_per_block + in_block;
    const bool here = u < total && token < a.num_tokens;
    const int w = u - in_block * per_token;
    const int h = w / per_head, j = w - h * per_head;
    const int kind = h < a.hq ? 0 : h < a.hq + a.hkv ? 1 : 2;  // q, k, v
    const int head = kind == 0 ? h : kind == 1 ? h - a.hq : h - a.hq - a.hkv;
    bool valid = here;
    int64_t slot = 0;
    if (here && kind != 0) {
      slot = __ldg(a.slots + token);
      if (slot < 0 || slot >= a.num_slots) {
        if (slot != -1 && kind == 2 && head == 0 && j == 0) pkv::raise_error(a.err, PKV_DERR_SLOT_RANGE);
        valid = false;
      }
    }
    int position = 0;
    if (kRope && here) {
      position = __ldg(a.positions + token);
      if (position < 0 || position >= a.max_position) {
        if (w == 0) pkv::raise_error(a.err, PKV_DERR_POSITION_RANGE);
        valid = false;
      }
    }
    int d0 = j * 8, d1 = a.head_dim / 2 + j * 8;
    const bool rotate = kRope && kind != 2 && j < turned;
    if (rotate) {
      d1 = a.rot_dim / 2 + j * 8;
    } else if (kRope && kind != 2) {
      d0 = a.rot_dim + (j - turned) * 8;
      d1 = d0 + (a.head_dim - a.rot_dim) / 2;
    }
    float x0[8] = {}, x1[8] = {};
    if (valid) {
      const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                     token * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) +
                     static_cast<int64_t>(head) * a.head_dim;
      load8(src + d0, x0);
      load8(src + d1, x1);
    }
    if (rotate && valid) {
      const float* row = a.cos_sin + static_cast<int64_t>(position) * a.rot_dim;
      const int half = a.rot_dim / 2;
      float c[8], s[8];
      if (!a.interleaved) {
        load8(row + j * 8, c);
        load8(row + half + j * 8, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y0 = turn<true>(x0[i], x1[i], c[i], s[i]);
          x1[i] = rounded<T>(turn<false>(x1[i], x0[i], c[i], s[i]));
          x0[i] = rounded<T>(y0);
        }
      } else {
        // pairs 4j .. 4j + 3 in the first run, rot_dim / 4 further on in the second
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = j * 4 + i * (half / 2);
          const float4 cv = __ldg(reinterpret_cast<const float4*>(row + at));
          const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half + at));
          c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
          s[4 * i] = sv.x, s[4 * i + 1] = sv.y, s[4 * i + 2] = sv.z, s[4 * i + 3] = sv.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y0 = turn<true>(x0[2 * i], x0[2 * i + 1], c[i], s[i]);
          x0[2 * i + 1] = rounded<T>(turn<false>(x0[2 * i + 1], x0[2 * i], c[i], s[i]));
          x0[2 * i] = rounded<T>(y0);
          const float y1 = turn<true>(x1[2 * i], x1[2 * i + 1], c[4 + i], s[4 + i]);
          x1[2 * i + 1] = rounded<T>(turn<false>(x1[2 * i + 1], x1[2 * i], c[4 + i], s[4 + i]));
          x1[2 * i] = rounded<T>(y1);
        }
      }
    }
    const float scale = kind == 2 ? a.v_scale : a.k_scale;
    if (kind == 0 && valid) {
      T* dst = static_cast<T*>(a.q_out) + (static_cast<int64_t>(token) * a.hq + head) * a.head_dim;
      store8(dst + d0, x0);
      store8(dst + d1, x1);
    }
    unsigned char* cache = kind == 2 ? a.v_cache : a.k_cache;
    store_cache<T, kFormat>(a, cache, slot, head, d0, x0, scale, valid && kind != 0);
    store_cache<T, kFormat>(a, cache, slot, head, d1, x1, scale, valid && kind != 0);
  }
}

template <typename T, Format kFormat, bool kRope>
int launch_store(const RopeArgs& a, cudaStream_t stream) {
  const int per_token = (a.hq + 2 * a.hkv) * (a.head_dim / 16);
  const int tokens = per_token >= 256 ? 1 : 256 / per_token;
  const unsigned grid = static_cast<unsigned>((a.num_tokens + tokens - 1) / tokens);
  return pkv::launch_pdl(kv_rope_store_kernel<T, kFormat, kRope>, dim3(grid), dim3(256), 0, stream, a, tokens) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

// One thread per group of 16: eight code bytes and a scale byte become 16 bf16.
__global__ void __launch_bounds__(256) kv_load_q4_kernel(uint4* __restrict__ k, uint4* __restrict__ v,
                                                         const unsigned char* __restrict__ k_cache,
                                                         const unsigned char* __restrict__ v_cache,
                                                         const int32_t* __restrict__ slots, int64_t total,
                                                         int groups, int64_t num_slots, int row_bytes, float k_scale,
                                                         float v_scale, unsigned int* err) {
  pkv::pdl_enter();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t token = i / (2 * groups);
    const int w = static_cast<int>(i - token * 2 * groups);
    const bool is_v = w >= groups;
    const int g = is_v ? w - groups : w;
    const int64_t slot = __ldg(slots + token);
    float f[16] = {};
    if (slot >= 0 && slot < num_slots) {
      const unsigned char* row = (is_v ? v_cache : k_cache) + slot * row_bytes;
      const uint2 codes = __ldg(reinterpret_cast<const uint2*>(row) + g);
      const float step = __fmul_rn(pkv::e4m3_value(__ldg(row + groups * 8 + g)), is_v ? v_scale : k_scale);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        f[j] = static_cast<float>(static_cast<int>((j < 8 ? codes.x : codes.y) >> (4 * (j & 7)) & 15u) - 8) * step;
    } else if (slot != -1 && w == 0) {
      pkv::raise_error(err, PKV_DERR_SLOT_RANGE);
    }
    uint4* dst = (is_v ? v : k) + (token * groups + g) * 2;
    dst[0] = Chunk<__nv_bfloat16>::pack(f);
    dst[1] = Chunk<__nv_bfloat16>::pack(f + 8);
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
  const int groups = num_kv_heads * head_dim / 16;
  const int64_t total = static_cast<int64_t>(num_tokens) * 2 * groups;
  const int64_t blocks = std::min<int64_t>((total + 255) / 256, static_cast<int64_t>(info.sms) * 8);
  return pkv::launch_pdl(kv_load_q4_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream,
                         static_cast<uint4*>(k), static_cast<uint4*>(v), static_cast<const unsigned char*>(k_cache),
                         static_cast<const unsigned char*>(v_cache), slot_mapping, total, groups,
                         static_cast<int64_t>(num_blocks) * block_size, pkv::q4_row_bytes(num_kv_heads, head_dim),
                         k_scale, v_scale, err) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}
