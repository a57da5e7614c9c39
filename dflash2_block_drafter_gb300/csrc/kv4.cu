// Rows of the 4-bit key/value cache of the drafter's attention sublayer, in and out (dflash2.ts #contextKV;
// MAX DFlash2Qwen3_5.materialize; kv4_attention.cu reads the cache).
//
// Quantisation, per token, head and group of 64 channels (affine, as dflash2.ts quantizedWeight's):
//   bias = bf16(min x), scale = bf16((max x - min x) / 15), code = clamp(round((x - bias) / scale), 0, 15)
// in IEEE fp32 with ties to even (scale = 0: code 0).
//
// A thread takes the same 16-byte chunk of K and of V of two tokens, all four loads in flight; a group's minimum
// and maximum are packed bf16 operations over eight lanes. 32768 tokens of 8 heads of 128 channels: 62 us in
// (2.8 TB/s), bound by issue slots (some 200 instructions a chunk, most of them the exact rounding of the
// quotients), and 32 us out (5.4 TB/s), bound by DRAM; 6 us for 16 tokens, both calls together.
#include <algorithm>

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
  int chunks, per_block;       // 16-byte chunks of a token's keys (and of its values); tokens of a CTA
  uint8_t* cache;
  __nv_bfloat16 *k_out, *v_out;
  int* err;
};

constexpr int kRowsThreads = 256;
constexpr int kRowsUnroll = 2;  // tokens of a thread in flight

// (A NaN is kept: it ends in its group's scale and bias, which then read as NaN.)
__device__ __forceinline__ uint32_t bf162_min(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmin2_nan(as_bf162(a), as_bf162(b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t bf162_max(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2_nan(as_bf162(a), as_bf162(b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Codes of eight values (pairs of bf16) of a group with minimum b and step s. The division is a product with
// the reciprocal, rounded by adding 2^23 + 2^22 and made exact afterwards: with d = x - b and n the
// rounded product, the residual d - n s comes from one FMA, and n moves by one where that is more than
// half a step (or half a step, and n odd): ties to even, as rounding the quotient gives. The values are
// bf16, so b is their exact minimum and n ends in [0, 15] (15 steps fall short of the range by less than
// half a step). The word is summed with the rounding constant still in every n, taken off at the end.
// A group with a NaN or an infinity, or a range past fp32, has s = NaN: word 0.
__device__ __forceinline__ uint32_t kv_quantise8(const uint32_t (&w)[4], float s, float b) {
  constexpr float kRound = 12582912.f;
  constexpr uint32_t kBits = 0x4b400000u;
  uint32_t word = 0;
  if (s >= 1.17549435e-38f) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const uint32_t past_half = __float_as_uint(0.5f * s) + 1u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = __uint_as_float((i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      const float d = x - b;
      const float m = fmaf(d, inv, kRound);
      const float r = fmaf(kRound - m, s, d);
      uint32_t n = __float_as_uint(m);
      const uint32_t rb = __float_as_uint(r);
      if ((rb & 0x7fffffffu) >= past_half - (n & 1u)) n += (static_cast<int>(rb) >> 31) | 1;
      word += n << (4 * i);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) word -= kBits << (4 * i);
  } else if (s > 0.f) {  // a subnormal step has no finite reciprocal
    for (int i = 0; i < 8; ++i) {
      const float x = __uint_as_float((i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      word |= static_cast<uint32_t>(fminf(fmaxf(rintf((x - b) / s), 0.f), 15.f)) << (4 * i);
    }
  }
  return word;
}

// Rows into slots (kRead: slots into rows). A thread takes one 16-byte chunk (8 channels) of the keys and the
// same one of the values of each of its tokens, two tokens in flight (what finds the slot is shared by
// both); eight lanes share a group of 64, whose minimum and (negated) maximum come from three shuffles of
// a pair. One pass over the rows; issue bounds the way in, the bytes the way out.
template <int D, bool kRead>
__global__ void __launch_bounds__(kRowsThreads) kv4_rows_kernel(const KvRowsArgs a) {
  using L = KvLayout<D>;
  pdl_trigger();
  pdl_wait();
  const int lane8 = threadIdx.x & 7;
  const uint32_t group = 0xffu << (threadIdx.x & 24);  // the group's eight lanes, which stay together
  // fewer chunks than threads: several tokens side by side
  const int rows = max(1, kRowsThreads / a.chunks), row = static_cast<int>(threadIdx.x) / a.chunks;
  const int granules = (1 << a.page_shift) / kKvGranule;
  const int page_bytes = a.heads * 2 * granules * L::kGranuleBytes;  // (heads, page size: below 2^31)
  const int to_values = granules * L::kGranuleBytes;
  const int64_t end = static_cast<int64_t>(a.num_pages) << a.page_shift;
  const int t_end = min(a.T, static_cast<int>(blockIdx.x + 1) * a.per_block);
  for (int x = a.chunks <= kRowsThreads ? threadIdx.x - row * a.chunks : threadIdx.x; x < a.chunks && row < rows;
       x += kRowsThreads) {
    const int col = x * 8, grp = col / kKvGroup % L::kGroups;
    uint8_t* base = a.cache + col / D * 2 * to_values;
    const int code_at = grp * (kKvGroup / 2) + lane8 * 4, par_at = L::kCodes + grp * 4;
    for (int t0 = static_cast<int>(blockIdx.x) * a.per_block + row; t0 < t_end; t0 += kRowsUnroll * rows) {
      uint8_t* g[kRowsUnroll];  // the keys' granule of the slot; null: not there
      int tok[kRowsUnroll];
#pragma unroll
      for (int u = 0; u < kRowsUnroll; ++u) {
        const int t = t0 + u * rows;
        int64_t slot = t < t_end ? a.slots[t] : -1;  // (an ordinary load: the kernel in front may have written it)
        if (slot >= end) {  // past the cache: recorded, skipped
          atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_BAD_INDEX));
          slot = -1;
        }
        const int in = static_cast<int>(slot) & ((1 << a.page_shift) - 1);
        tok[u] = in % kKvGranule;
        g[u] = slot < 0 ? nullptr
                        : base + (static_cast<int64_t>(static_cast<int>(slot >> a.page_shift)) * page_bytes +
                                  in / kKvGranule * L::kGranuleBytes);
      }
      if (kRead) {
        uint32_t code[kRowsUnroll][2], par[kRowsUnroll][2];
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u) {
          code[u][0] = code[u][1] = par[u][0] = par[u][1] = 0u;
          if (g[u] == nullptr) continue;
          const uint8_t *c = g[u] + code_at + tok[u] * L::kRow, *p = g[u] + par_at + tok[u] * L::kGroups * 4;
          code[u][0] = *reinterpret_cast<const uint32_t*>(c);
          code[u][1] = *reinterpret_cast<const uint32_t*>(c + to_values);
          par[u][0] = *reinterpret_cast<const uint32_t*>(p);
          par[u][1] = *reinterpret_cast<const uint32_t*>(p + to_values);
        }
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u) {
          const int t = t0 + u * rows;
          if (t >= t_end) continue;
          const int64_t at = static_cast<int64_t>(t) * (a.heads * D) + col;
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const __nv_bfloat162 sb = as_bf162(par[u][side]);
            const __nv_bfloat162 s2 = __low2bfloat162(sb), b2 = __high2bfloat162(sb);
            uint32_t p[4];  // channels (i, i + 4); zeros for a slot that is not there
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = kv_value(code[u][side] >> (4 * i), s2, b2);
            *reinterpret_cast<uint4*>((side == 0 ? a.k_out : a.v_out) + at) =
                make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                           __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
          }
        }
      } else {
        uint4 raw[kRowsUnroll][2];
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u) {
          raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
          if (g[u] == nullptr) continue;
          raw[u][0] = __ldg(reinterpret_cast<const uint4*>(a.k + (t0 + u * rows) * a.k_stride + col));
          raw[u][1] = __ldg(reinterpret_cast<const uint4*>(a.v + (t0 + u * rows) * a.v_stride + col));
        }
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u) {
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const uint4 v = raw[u][side];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            const uint32_t lo2 = bf162_min(bf162_min(w[0], w[1]), bf162_min(w[2], w[3]));
            const uint32_t hi2 = bf162_max(bf162_max(w[0], w[1]), bf162_max(w[2], w[3])) ^ 0x80008000u;
            uint32_t m = bf162_min(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));  // (minimum, - maximum)
#pragma unroll
            for (int i = 1; i < 8; i <<= 1) m = bf162_min(m, __shfl_xor_sync(group, m, i));
            if (g[u] == nullptr) continue;
            const float lo = __uint_as_float(m << 16), hi = -__uint_as_float(m & 0xffff0000u);
            // (hi - lo) / 15 correctly rounded: a product and one correction by its residual (P. Markstein's
            // method); NaN for a range that is not finite
            const float range = hi - lo, q0 = range * (1.f / 15.f);
            const float q = fmaf(fmaf(-15.f, q0, range), 1.f / 15.f, q0);
            const __nv_bfloat16 scale = __float2bfloat16_rn(q);
            uint8_t* to = g[u] + (side == 0 ? 0 : to_values);
            *reinterpret_cast<uint32_t*>(to + code_at + tok[u] * L::kRow) = kv_quantise8(w, __bfloat162float(scale), lo);
            if (lane8 == 0)
              *reinterpret_cast<uint32_t*>(to + par_at + tok[u] * L::kGroups * 4) =
                  (m << 16) | static_cast<uint32_t>(__bfloat16_as_ushort(scale));
          }
        }
      }
    }
  }
}

template <int D>
int launch_rows(KvRowsArgs a, bool read, cudaStream_t st) {
  a.chunks = a.heads * (D / 8);
  // tokens of a CTA: two to a thread, unless that leaves SMs without a CTA
  const int most = kRowsUnroll * std::max(1, kRowsThreads / a.chunks);
  a.per_block = std::max(1, std::min(most, a.T / (2 * sm_count())));
  const cudaError_t e = launch_pdl(read ? kv4_rows_kernel<D, true> : kv4_rows_kernel<D, false>,
                                   dim3(static_cast<unsigned>((a.T + a.per_block - 1) / a.per_block)), dim3(kRowsThreads),
                                   0, st, nullptr, 0, a);
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
