// The 4-bit cache format.
//
// A token's K (or V) row: for each KV head head_dim / 2 code bytes (byte i holds
// the codes of elements 2i, low nibble, and 2i + 1), then for each KV head
// head_dim / 16 scale bytes (E4M3, one per 16 elements), then zeros up to a
// multiple of 16 bytes, so that every row can be copied by the TMA engine
// whatever the number of heads.  An element is (code - 8) * scale * T with one
// float T per tensor.
//
// E4M3 scales over 16 elements: (code - 8) * scale has at most 7 significant
// bits, so f16 (and bf16) hold it exactly and the attention kernels' products
// see the cached values themselves.
#pragma once

#include "common.cuh"

namespace pkv {

__host__ __device__ constexpr int q4_scale_offset(int hkv, int head_dim) { return hkv * (head_dim / 2); }
__host__ __device__ constexpr int q4_row_bytes(int hkv, int head_dim) {
  return (hkv * (head_dim / 2 + head_dim / 16) + 15) / 16 * 16;
}
inline bool q4_head_dim(int head_dim) { return head_dim == 64 || head_dim == 128; }

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_keep_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// E4M3 code of x (low byte), round to nearest even, saturating; a NaN keeps its code.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const uint32_t h = e4m3x2_to_f16x2(code & 0xffu);
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// Eight codes (element i in bits 4i) of x[i] / (scale * T); all 8 (the value 0)
// where that step is 0 or NaN.
__device__ __forceinline__ uint32_t q4_codes8(const float (&x)[8], uint32_t scale_code, float tensor_scale) {
  const float step = __fmul_rn(e4m3_value(scale_code), tensor_scale);
  uint32_t w = 0x88888888u;
  if (step > 0.f) {
    w = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = fminf(fmaxf(rintf(__fdiv_rn(x[i], step)), -8.f), 7.f);
      w |= static_cast<uint32_t>(static_cast<int>(r) + 8) << (4 * i);
    }
  }
  return w;
}

// Codes to matrix operands.  A word of eight codes becomes four f16 pairs with two
// shifts, four and-ors and four fmas: a nibble n in mantissa bits 9..6 under the
// exponent of 4 is the number 4 + n / 4, in bits 5..2 under the exponent of 64 it is
// 64 + n / 4, and x s - 6 s (or - 66 s) is (n - 8) s / 4.  Every step is exact:
// (n - 8) s has 7 significant bits, 66 s at most 9 and stays below f16's end.
// (Conversion instructions run at 16 results per clock and SM.)
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// A scale pair with what the two nibble positions subtract.
struct Q4Scale {
  uint32_t s, low, high;
  __device__ __forceinline__ explicit Q4Scale(uint32_t pair)
      : s(pair), low(hmul2(pair, 0xc600c600u)), high(hmul2(pair, 0xd420d420u)) {}
};
// The four f16 pairs of a word: nibbles (0, 4), (1, 5), (2, 6) and (3, 7), as (n - 8) / 4 times the scale pair.
__device__ __forceinline__ void widen_q4(uint32_t w, const Q4Scale& k, uint32_t (&f)[4]) {
  const uint32_t y0 = w << 2, y1 = w >> 6;
  f[0] = hfma2((y0 & 0x003c003cu) | 0x54005400u, k.s, k.high);
  f[1] = hfma2((y0 & 0x03c003c0u) | 0x44004400u, k.s, k.low);
  f[2] = hfma2((y1 & 0x003c003cu) | 0x54005400u, k.s, k.high);
  f[3] = hfma2((y1 & 0x03c003c0u) | 0x44004400u, k.s, k.low);
}

}  // namespace pkv
