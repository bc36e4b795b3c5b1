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

}  // namespace pkv
