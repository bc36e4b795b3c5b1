// The 4-bit cache format.
//
// A token's K (or V) row: for each KV head head_dim / 2 code bytes (byte i holds
// the codes of elements 2i, low nibble, and 2i + 1), then for each KV head
// head_dim / 16 scale bytes (E4M3, one per 16 elements), then unused bytes, which
// no store writes, up to a multiple of 16, so that every row can be copied by the
// TMA engine whatever the number of heads.  An element is (code - 8) * scale * T with one
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
// Tensor scales the attention calls take: unnormalized sums of weighted values times one stay in float32.
inline bool q4_attention_scale(float t) { return t >= 0x1p-64f && t <= 0x1p64f; }
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

// Two-lane fp32 arithmetic.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// x / d rounded to float32, from inv, the rounded reciprocal of d: Markstein's
// theorem (IBM J. Res. Dev. 34, 1990) makes one correction by the exact remainder
// of a quotient that is off by less than a unit in the last place the rounded
// one, as long as neither leaves the normal numbers.
__device__ __forceinline__ uint64_t quotient2(uint64_t x, float d, float inv) {
  const uint64_t i2 = pair(inv, inv), q = mul2(x, i2);
  return fma2(fma2(q, pair(-d, -d), x), i2, q);
}
// Whether a divisor leaves room for that: x up to 2^40 times larger or smaller.
__device__ __forceinline__ bool divides(float d) { return d >= 0x1p-80f && d <= 0x1p80f; }

// Eight codes (element i in bits 4i) of x[i] / (scale * T), the quotient rounded to
// float32 and then to the nearest even whole number; all 8 (the value 0) where that
// step is 0 or NaN.  Ties are common (of every 32 bf16 values between two codes one
// is the middle), so the quotient has to be the rounded one.  A normal scale that
// did not saturate keeps it below 7.5, so nothing is cut off.  Adding 1.5 2^23 + 8
// rounds to a whole number and leaves the code in the low bits.
__device__ __forceinline__ uint32_t q4_codes8(const float (&x)[8], uint32_t scale_code, float tensor_scale) {
  const float step = __fmul_rn(e4m3_value(scale_code), tensor_scale);
  uint32_t w = 0u;
  if (scale_code >= 0x08u && scale_code < 0x7eu && divides(step)) {
    const float inv = __frcp_rn(step);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float a, b;
      split(fma2(quotient2(pair(x[i], x[i + 1]), step, inv), pair(1.f, 1.f), pair(12582920.f, 12582920.f)), a, b);
      w += __float_as_uint(a) << (4 * i);
      w += __float_as_uint(b) << (4 * i + 4);
    }
    return w - 0x4b400000u * 0x11111111u;
  }
  if (!(step > 0.f)) return 0x88888888u;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const float r = fminf(fmaxf(rintf(__fdiv_rn(x[i], step)), -8.f), 7.f);
    w |= static_cast<uint32_t>(static_cast<int>(r) + 8) << (4 * i);
  }
  return w;
}

// Eight E4M3 codes of x[i] / scale (rounded to float32 first), saturating; a NaN keeps its code.
__device__ __forceinline__ uint2 e4m3_codes8(const float (&x)[8], float scale) {
  float y[8];
  bool exact = divides(scale);
  if (exact) {
    const float inv = __frcp_rn(scale);
    uint64_t nan = 0ull;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t q = quotient2(pair(x[i], x[i + 1]), scale, inv);
      nan = fma2(q, 0ull, nan);
      split(q, y[i], y[i + 1]);
      y[i] = copysignf(y[i], x[i]);  // (the correction of a zero loses its sign)
      y[i + 1] = copysignf(y[i + 1], x[i + 1]);
    }
    float n0, n1;
    split(nan, n0, n1);
    exact = n0 + n1 == 0.f;  // (infinities, and quotients that overflowed, end as NaN)
  }
  if (!exact) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], scale);
  }
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y[2 * i + 1]), "f"(y[2 * i]));
    c[i] = r;
  }
  return make_uint2(prmt(c[0], c[1], 0x5410u), prmt(c[2], c[3], 0x5410u));
}

// E4M3 code of a group's scale, its largest magnitude over 7 T.
__device__ __forceinline__ uint32_t q4_scale_code(float top, float tensor_scale) {
  return to_e4m3(__fdiv_rn(top, __fmul_rn(7.f, tensor_scale)));
}

// Codes to matrix operands, small integers made floats by putting their bits under a
// constant exponent.  A word of eight codes becomes four f16 pairs with one
// shift, four and-ors and four fmas: a nibble n in mantissa bits 3..0 under the
// exponent of 16 is the number 16 + n / 64, in bits 7..4 under the exponent of 1 it is
// 1 + n / 64, and x s - 16.125 s (or - 1.125 s) is (n - 8) s / 64.  Every step is
// exact: (n - 8) s has 7 significant bits, 16.125 s 11, and s / 64 is a whole multiple of
// f16's least number.  (Conversion instructions run at 16 results per clock and SM.)
constexpr float kQ4Unit = 64.f;  // what the widened values are to be multiplied by
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
      : s(pair), low(hmul2(pair, 0xcc08cc08u)), high(hmul2(pair, 0xbc80bc80u)) {}
};
// (a & b) | c
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// The four f16 pairs of a word: nibbles (0, 4), (1, 5), (2, 6) and (3, 7), as (n - 8) / 64 times the scale pair.
__device__ __forceinline__ void widen_q4(uint32_t w, const Q4Scale& k, uint32_t (&f)[4]) {
  uint32_t y;
  asm("shr.u32 %0, %1, 8;" : "=r"(y) : "r"(w));
  f[0] = hfma2(and_or(w, 0x000f000fu, 0x4c004c00u), k.s, k.low);
  f[1] = hfma2(and_or(w, 0x00f000f0u, 0x3c003c00u), k.s, k.high);
  f[2] = hfma2(and_or(y, 0x000f000fu, 0x4c004c00u), k.s, k.low);
  f[3] = hfma2(and_or(y, 0x00f000f0u, 0x3c003c00u), k.s, k.high);
}

}  // namespace pkv
