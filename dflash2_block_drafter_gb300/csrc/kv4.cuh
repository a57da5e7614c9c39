// Layout and arithmetic of the 4-bit key/value cache, shared by its writer and its readers.
//
// The cache is [num_pages][heads][2 sides][page_size / 16] granules. A granule holds 16 tokens of one
// head and side: first their codes, [16][D / 2] bytes (code of channel d in bits 4 (d % 8) .. of the
// token's 32-bit word d / 8), then their parameters, [16][D / 64] pairs of bf16 (scale, bias). A
// reader therefore fetches 16 tokens with one bulk copy, whatever the page size (a multiple of 16).
// The value of a code is scale * code + bias.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

namespace dfl {

constexpr int kKvGroup = 64;    // channels that share a scale and a bias
constexpr int kKvGranule = 16;  // tokens per granule

template <int D>
struct KvLayout {
  static constexpr int kGroups = D / kKvGroup;
  static constexpr int kRow = D / 2;                               // code bytes of a token
  static constexpr int kCodes = kKvGranule * kRow;                 // code bytes of a granule
  static constexpr int kGranuleBytes = kCodes + kKvGranule * kGroups * 4;
};

// Codes of channels i and i + 4 of a word as an exact bf16 pair (128 + code): 0x4300 | n is 128 + n.
// `w` is the word shifted right by 4 i.
__device__ __forceinline__ __nv_bfloat162 kv_codes(uint32_t w) {
  const uint32_t u = (w & 0x000F000Fu) | 0x43004300u;
  return *reinterpret_cast<const __nv_bfloat162*>(&u);
}
// scale * code + bias of such a pair, rounded once to bf16 (128 + code - 128 is exact).
__device__ __forceinline__ uint32_t kv_value(uint32_t w, __nv_bfloat162 scale, __nv_bfloat162 bias) {
  const __nv_bfloat162 k128 = __halves2bfloat162(__ushort_as_bfloat16(0x4300), __ushort_as_bfloat16(0x4300));
  const __nv_bfloat162 v = __hfma2(scale, __hsub2(kv_codes(w), k128), bias);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); }

}  // namespace dfl
