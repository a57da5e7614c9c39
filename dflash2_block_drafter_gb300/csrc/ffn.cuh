// Device arithmetic shared by the gated feed-forward kernels (ffn.cu, ffn_small.cu).
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "dflash2.h"

namespace dfl {

__device__ __forceinline__ float logistic(float w) { return __fdividef(1.f, 1.f + __expf(-w)); }
// s(w(g)) and w'(g): act(g) = g s, act'(g) = s + g s (1 - s) w'.
__device__ __forceinline__ float ffn_gate(float g, int act, float& slope) {
  if (act == DFLASH2_ACT_SILU) {
    slope = 1.f;
    return logistic(g);
  }
  constexpr float k = 1.5957691216057308f;  // 2 sqrt(2 / pi)
  const float g2 = g * g;
  slope = k * fmaf(3.f * 0.044715f, g2, 1.f);
  return logistic(k * g * fmaf(0.044715f, g2, 1.f));
}
// The kept products: g and u of one channel in a 32-bit word, 16 bits each: sign, 6 exponent bits (bias
// 31), 9 mantissa bits. The gradients see g and u through dg and du, which are themselves rounded to
// bf16 (8 significant bits): with bf16 here too the roundings add up (relative rms error of dx and dW
// 0.0031 against 0.0017 for a rounded exact result); 10 significant bits leave 0.0024, what dg's own
// rounding costs, for the same bytes. Magnitudes from 2^-30 to 2^32 keep their 10 bits, smaller ones
// go down to steps of 2^-39, larger ones saturate. Exponent 63 is infinity (mantissa 0) or NaN, as in the wider
// formats, so that gradients of a product that is not finite say so; both read as NaN (two multiplications
// instead of a comparison and a selection: 0.3 % of 1001 x 2568 x 6920 with gradients instead of 0.7 %).
__device__ __forceinline__ uint32_t ffn_keep1(float x) {
  const uint32_t u = __float_as_uint(x * 1.262177448e-29f);  // 2^-96: the exponent fits 6 bits
  const uint32_t m = u & 0x7fffffffu, t = m >> 14;
  const uint32_t h = min((m + 0x1fffu + (t & 1u)) >> 14, 0x7dffu);  // ties to even; 2^32 (1 - 2^-10) at most
  return ((m < 0x7f800000u ? h : t) & 0x7fffu) | ((u >> 16) & 0x8000u);
}
__device__ __forceinline__ uint32_t ffn_keep(float g, float u) { return ffn_keep1(g) | (ffn_keep1(u) << 16); }
__device__ __forceinline__ float ffn_kept1(uint32_t h) {
  const float y = __uint_as_float(((h & 0x8000u) << 16) | ((h & 0x7fffu) << 14)) * 7.922816251e28f;  // 2^96
  return fmaf(y * 7.922816251e28f, 0.f, y);  // exponent 63 passes fp32's range: infinity times 0
}

__device__ __forceinline__ uint32_t ffn_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace dfl
