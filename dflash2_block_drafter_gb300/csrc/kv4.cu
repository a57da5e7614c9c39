// Rows of the 4-bit key/value cache of the drafter's attention sublayer, in and out (dflash2.ts #contextKV;
// MAX DFlash2Qwen3_5.materialize; kv4_attention.cu reads the cache).
//
// Quantisation, per token, head and group of 64 channels (affine, as dflash2.ts quantizedWeight's):
//   bias = bf16(min x), scale = bf16((max x - min x) / 15), code = clamp(round((x - bias) / scale), 0, 15)
// in IEEE fp32 with ties to even (scale = 0: code 0).
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace dfl {
namespace {

// ---------------------------------------------------------------- rows in and out of the cache
struct KvRowsArgs {
  const __nv_bfloat16 *k, *v;
  int64_t k_stride, v_stride;  // elements between rows
  const int64_t* slots;
  int T, heads, page_shift, num_pages;
  uint8_t* cache;
  __nv_bfloat16 *k_out, *v_out;
  int* err;
};

// The granule of a slot, or null (a negative slot: skipped; one past the cache: recorded, skipped).
template <int D>
__device__ __forceinline__ uint8_t* kv_slot(const KvRowsArgs& a, int64_t slot, int head, int side, int& token) {
  if (slot < 0) return nullptr;
  const int64_t page = slot >> a.page_shift;
  if (page >= a.num_pages) {
    atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_BAD_INDEX));
    return nullptr;
  }
  const int in = static_cast<int>(slot & ((1 << a.page_shift) - 1));
  const int granules = (1 << a.page_shift) / kKvGranule;
  token = in % kKvGranule;
  return a.cache + (((page * a.heads + head) * 2 + side) * granules + in / kKvGranule) *
                       static_cast<int64_t>(KvLayout<D>::kGranuleBytes);
}

// Eight lanes per group of 64 channels: lane i loads channels 8 i .. 8 i + 7 (16 bytes), the group's
// minimum and maximum come from three shuffles, and each lane stores one word of codes. One pass over
// the rows, so the bytes bound it. Blocks walk (token, side, head, group) in memory order of the rows.
template <int D, bool kRead>
__global__ void __launch_bounds__(256) kv4_rows_kernel(const KvRowsArgs a) {
  pdl_trigger();
  pdl_wait();
  using L = KvLayout<D>;
  const int lane8 = threadIdx.x & 7;
  const int per_side = a.heads * L::kGroups;
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 3;
  const int64_t items = static_cast<int64_t>(a.T) * 2 * per_side;
  const bool in_range = item < items;
  const int64_t it = in_range ? item : 0;
  const int t = static_cast<int>(it / (2 * per_side));
  const int rest = static_cast<int>(it - static_cast<int64_t>(t) * 2 * per_side);
  const int side = rest / per_side;
  const int head = (rest - side * per_side) / L::kGroups;
  const int grp = rest % L::kGroups;
  const int col = head * D + grp * kKvGroup + lane8 * 8;
  int token = 0;
  uint8_t* gran = in_range ? kv_slot<D>(a, a.slots[t], head, side, token) : nullptr;
  const int code_at = token * L::kRow + grp * (kKvGroup / 2) + lane8 * 4;
  const int par_at = L::kCodes + (token * L::kGroups + grp) * 4;
  if (kRead) {
    if (!in_range) return;
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (gran != nullptr) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(gran + code_at);
      const uint32_t par = *reinterpret_cast<const uint32_t*>(gran + par_at);
      const __nv_bfloat162 sb = as_bf162(par);
      const __nv_bfloat162 s2 = __low2bfloat162(sb), b2 = __high2bfloat162(sb);
      uint32_t p[4];  // channels (i, i + 4)
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = kv_value(w >> (4 * i), s2, b2);
      o.x = __byte_perm(p[0], p[1], 0x5410);
      o.y = __byte_perm(p[2], p[3], 0x5410);
      o.z = __byte_perm(p[0], p[1], 0x7632);
      o.w = __byte_perm(p[2], p[3], 0x7632);
    }
    __nv_bfloat16* out = side == 0 ? a.k_out : a.v_out;
    *reinterpret_cast<uint4*>(out + static_cast<int64_t>(t) * a.heads * D + col) = o;
    return;
  }
  float x[8] = {};
  if (gran != nullptr) {
    const __nv_bfloat16* src = side == 0 ? a.k + t * a.k_stride : a.v + t * a.v_stride;
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + col));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(as_bf162(w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  if (gran == nullptr) return;
  const __nv_bfloat16 scale = __float2bfloat16_rn((hi - lo) / 15.f);
  const __nv_bfloat16 bias = __float2bfloat16_rn(lo);
  const float s = __bfloat162float(scale), b = __bfloat162float(bias);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = s > 0.f ? fminf(fmaxf(rintf((x[i] - b) / s), 0.f), 15.f) : 0.f;
    word |= static_cast<uint32_t>(c) << (4 * i);
  }
  *reinterpret_cast<uint32_t*>(gran + code_at) = word;
  if (lane8 == 0) {
    const __nv_bfloat162 sb = __halves2bfloat162(scale, bias);
    *reinterpret_cast<__nv_bfloat162*>(gran + par_at) = sb;
  }
}

template <int D>
int launch_rows(const KvRowsArgs& a, bool read, cudaStream_t st) {
  const int64_t threads = static_cast<int64_t>(a.T) * 2 * a.heads * KvLayout<D>::kGroups * 8;
  const int64_t blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffffLL) return fail(DFLASH2_ERR_INVALID_ARG, "T=%d rows are too many for one call", a.T);
  const cudaError_t e = launch_pdl(read ? kv4_rows_kernel<D, true> : kv4_rows_kernel<D, false>,
                                   dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, nullptr, 0, a);
  return e == cudaSuccess ? DFLASH2_OK : fail(DFLASH2_ERR_CUDA, "cache row launch failed: %s", cudaGetErrorString(e));
}

int log2_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

}  // namespace

int launch_kv4_rows(const Kv4Rows& r, cudaStream_t st) {
  KvRowsArgs a{};
  a.k = static_cast<const __nv_bfloat16*>(r.k);
  a.v = static_cast<const __nv_bfloat16*>(r.v);
  a.k_stride = r.k_stride;
  a.v_stride = r.v_stride;
  a.slots = r.slots;
  a.T = r.T;
  a.heads = r.heads;
  a.page_shift = log2_of(r.page_size);
  a.num_pages = r.num_pages;
  a.cache = static_cast<uint8_t*>(r.cache);
  a.k_out = static_cast<__nv_bfloat16*>(r.k_out);
  a.v_out = static_cast<__nv_bfloat16*>(r.v_out);
  a.err = device_error_word();
  if (a.err == nullptr) return fail(DFLASH2_ERR_CUDA, "no device error word");
  const bool read = r.k_out != nullptr;
  return r.D == 64 ? launch_rows<64>(a, read, st) : launch_rows<128>(a, read, st);
}

}  // namespace dfl
