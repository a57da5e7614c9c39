// Candidates from logits: penalties for repeated tokens, token biases and a grammar mask applied to each row, the K
// best tokens, and the adjusted logits where they are wanted.
//
// Row m of request b, token v, with c the times that v was generated (in the request's history after its prompt, or
// by a drafted row on m's line of ancestors, m itself among them):
//   y = x > 0 ? x / repetition : x * repetition   if v was generated or stands in the prompt
//   y = y - (frequency * c + presence)            if c > 0
//   y = y + bias                                  if the request's list has v (its first entry)
//   y = -inf                                      if the mask's bit v is clear
// each step rounded to fp32, so that the order of nearly equal tokens is defined to the last bit.
//
// The work is one read of the logits. A cluster of CTAs shares a row, each CTA a slice of the vocabulary (16384 tokens
// at most: 64 a thread, which stay in registers between the two looks at them), and works through a range of rows.
// What applies to few tokens does not burden the rest: the tokens that the history, the drafted rows and the biases
// name are collected once for all of a request's rows (a bit a token in shared memory; its rank among the set bits
// finds its counter), computed apart from the stream, and only left out of it there.
//
// The K best of a slice: the K-th largest of sixteen groups' maxima bounds the K-th largest value from below, so the
// few values that reach it are listed and ranked against each other by (value, lower token). A list that overflows (a
// row whose large values lie in few threads' hands) is replaced by K rounds of a maximum. Only what is above -inf is
// listed; rows with fewer than K such tokens are filled with the lowest of the others. The cluster's lists are merged
// through distributed shared memory, a chunk of rows at a time.
#include <algorithm>

#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"
#include "tree.cuh"
#include "warp_keys.cuh"

namespace dfl {
namespace {

constexpr int kPickThreads = 256, kPickWarps = kPickThreads / 32;
constexpr int kPickElems = 64;                             // tokens a thread holds
constexpr int kPickSlice = kPickThreads * kPickElems;
constexpr int kPickRows = 32;                              // rows a chunk
constexpr int kPickList = 1024;
constexpr int kPickK = 16;
constexpr uint32_t kCountMask = (1u << 20) - 1, kInPrompt = 1u << 20;  // a counter; over it, which bias
constexpr int kBiasShift = 21;

struct PickArgs {
  LogitsTopk r;
  int cluster, slice, subs, cap;  // CTAs a row, tokens a CTA, how often; counters that fit
  int* err;
};

struct PickShared {
  unsigned long long list[kPickList];
  unsigned long long best[kPickRows][kPickK];  // (key, ~token), best first; 0: none
  uint64_t line[kPickRows];                    // the row's drafted ancestors
  unsigned long long red[kPickWarps];
  int request[kPickRows], first[kPickRows], state[kPickRows];  // 0: no row of any request, 1: a row, 2: not there
  uint32_t bits[kPickSlice / 32];
  uint32_t group_max[16];
  int count[2];
  int warp_sum[kPickWarps];
  uint16_t base[kPickSlice / 32];
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// An order-preserving key; NaN above every number (and an entry of it below all ones).
constexpr uint32_t kKeyNan = 0xfffffffeu;
__device__ __forceinline__ uint32_t pick_key(float v) { return v != v ? kKeyNan : float_key(v); }
__device__ __forceinline__ float pick_value(uint32_t k) { return k == kKeyNan ? __uint_as_float(0x7fffffffu) : key_float(k); }
__device__ __forceinline__ unsigned long long pick_entry(float v, int token) {
  return (static_cast<unsigned long long>(pick_key(v)) << 32) | static_cast<uint32_t>(~token);
}

// Sixteen bytes of logits.
template <typename T>
struct PickVec;
template <>
struct PickVec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ float get(const uint4& u, int j) {
    return __uint_as_float(j == 0 ? u.x : (j == 1 ? u.y : (j == 2 ? u.z : u.w)));
  }
  // elements whose bit is set become -inf
  static __device__ __forceinline__ void drop(uint4& u, uint32_t bits) {
    if (bits & 1u) u.x = 0xff800000u;
    if (bits & 2u) u.y = 0xff800000u;
    if (bits & 4u) u.z = 0xff800000u;
    if (bits & 8u) u.w = 0xff800000u;
  }
  static __device__ __forceinline__ float max(const uint4& u) {
    return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)), max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  static __device__ __forceinline__ uint4 load_some(const float* p, int n) {
    uint4 u;
    u.x = n > 0 ? __float_as_uint(p[0]) : 0xff800000u;
    u.y = n > 1 ? __float_as_uint(p[1]) : 0xff800000u;
    u.z = n > 2 ? __float_as_uint(p[2]) : 0xff800000u;
    u.w = n > 3 ? __float_as_uint(p[3]) : 0xff800000u;
    return u;
  }
  static __device__ __forceinline__ void store_some(float* p, const uint4& u, int n) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = get(u, j);
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};
template <>
struct PickVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ uint32_t word(const uint4& u, int i) {
    return i == 0 ? u.x : (i == 1 ? u.y : (i == 2 ? u.z : u.w));
  }
  static __device__ __forceinline__ float get(const uint4& u, int j) {
    const uint32_t w = word(u, j >> 1);
    return __uint_as_float((j & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ uint32_t drop2(uint32_t w, uint32_t bits) {
    if (bits & 1u) w = (w & 0xffff0000u) | 0xff80u;
    if (bits & 2u) w = (w & 0xffffu) | 0xff800000u;
    return w;
  }
  static __device__ __forceinline__ void drop(uint4& u, uint32_t bits) {
    u.x = drop2(u.x, bits);
    u.y = drop2(u.y, bits >> 2);
    u.z = drop2(u.z, bits >> 4);
    u.w = drop2(u.w, bits >> 6);
  }
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  static __device__ __forceinline__ float max(const uint4& u) {
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(two(u.x), two(u.y)), __hmax2_nan(two(u.z), two(u.w)));
    return max_nan(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ uint4 load_some(const __nv_bfloat16* p, int n) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < n ? reinterpret_cast<const unsigned short*>(p)[2 * i] : 0xff80u;
      const uint32_t hi = 2 * i + 1 < n ? reinterpret_cast<const unsigned short*>(p)[2 * i + 1] : 0xff80u;
      w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void store_some(__nv_bfloat16* p, const uint4& u, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) reinterpret_cast<unsigned short*>(p)[j] = static_cast<unsigned short>(word(u, j >> 1) >> (16 * (j & 1)));
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};

__device__ __forceinline__ unsigned long long max_u64(unsigned long long a, unsigned long long b) { return a > b ? a : b; }
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<unsigned long long>(hi) << 32) | lo;
}
__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads, 2) logits_topk_kernel(const PickArgs a) {
  using Vec = PickVec<T>;
  constexpr int kN = Vec::kN, kGroups = kPickElems / kN;
  constexpr uint32_t kAll = (1u << kN) - 1;
  __shared__ PickShared s;
  extern __shared__ __align__(16) uint8_t pick_smem[];
  uint32_t* words = reinterpret_cast<uint32_t*>(pick_smem);       // [cap] counters of the named tokens
  float* vals = reinterpret_cast<float*>(words + a.cap);          // [cap] their adjusted values
  uint16_t* offs = reinterpret_cast<uint16_t*>(vals + a.cap);     // [cap] their places in the slice
  const LogitsTopk& r = a.r;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cluster = static_cast<int>(blockIdx.x) / a.cluster, clusters = static_cast<int>(gridDim.x) / a.cluster;
  const int row0 = static_cast<int>(static_cast<long long>(r.M) * cluster / clusters);
  const int row1 = static_cast<int>(static_cast<long long>(r.M) * (cluster + 1) / clusters);
  const bool named = a.cap > 0;
  pdl_trigger();
  pdl_wait();
  auto record = [&](int status) { atomicCAS(a.err, 0, status); };
  if (blockIdx.x == 0 && r.row_off != nullptr)
    for (int b = tid; b < r.B; b += kPickThreads) {
      const int lo = __ldg(r.row_off + b), hi = __ldg(r.row_off + b + 1);
      if (lo < 0 || hi < lo || hi > r.M) record(DFLASH2_ERR_INVALID_ARG);
    }
  const int each = r.row_off == nullptr ? r.M / r.B : 0;
  int turn = 0;

  for (int c0 = row0; c0 < row1; c0 += kPickRows) {
    const int rows = min(kPickRows, row1 - c0);
    // ---- the chunk's rows: their requests and lines of ancestors
    if (tid < rows) {
      const int m = c0 + tid;
      int b, first, state = 1;
      if (each > 0) {
        b = m / each;
        first = b * each;
      } else {
        int lo = 0, hi = r.B - 1;  // the last request that starts at or before the row
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (__ldg(r.row_off + mid) <= m)
            lo = mid;
          else
            hi = mid - 1;
        }
        b = lo;
        first = __ldg(r.row_off + b);
        if (first < 0 || first > m || m >= __ldg(r.row_off + b + 1)) state = 0;
      }
      if (state == 1 && r.tokens != nullptr && m - first >= kTreeRows) {
        record(DFLASH2_ERR_INVALID_ARG);
        state = 0;
      }
      s.request[tid] = b;
      s.first[tid] = first;
      s.state[tid] = state;
      s.line[tid] = (2ull << min(max(m - first, 0), kTreeRows - 1)) - 1;  // (without parents: every row before it)
    }
    __syncthreads();
    if (r.tokens != nullptr && r.parents != nullptr) {
      int heads = 0;
      for (int i = 0; i < rows; ++i) {
        if (s.state[i] == 0 || (i > 0 && s.state[i - 1] != 0 && s.request[i - 1] == s.request[i])) continue;
        if ((heads++ & (kPickWarps - 1)) != warp) continue;
        const int b = s.request[i], first = s.first[i];
        const int all = each > 0 ? each : min(__ldg(r.row_off + b + 1), r.M) - first;
        int parent[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) parent[h] = lane + 32 * h < all ? __ldg(r.parents + first + lane + 32 * h) : -2;
        bool bad;
        const TreeLines tree = tree_lines(parent, min(all, kTreeRows), bad);
        if (bad) record(DFLASH2_ERR_BAD_INDEX);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = first + lane + 32 * h - c0;
          if (at >= i && at < rows && s.state[at] == 1 && s.request[at] == b) s.line[at] = tree.line[h];
        }
      }
      __syncthreads();
      if (tid < rows && s.state[tid] == 1 && s.line[tid] == 0ull) s.state[tid] = 2;
      __syncthreads();
    }

    for (int sub = 0; sub < a.subs; ++sub) {
      const int lo = (sub * a.cluster + rank) * a.slice;
      const int wlen = max(0, min(a.slice, r.V - lo));
      for (int i0 = 0; i0 < rows;) {
        // ---- rows [i0, i1) of one request
        const int b = s.request[i0];
        int i1 = i0 + 1;
        while (i1 < rows && s.request[i1] == b && s.state[i1] != 0 && s.state[i0] != 0) ++i1;
        const int seg0 = i0;
        i0 = i1;
        if (s.state[seg0] == 0) continue;
        const int first = s.first[seg0];
        int n = 0;  // named tokens of the slice
        auto rank_of = [&](int u) { return s.base[u >> 5] + __popc(s.bits[u >> 5] & ((1u << (u & 31)) - 1u)); };
        if (named) {
          const int32_t* hist = r.history != nullptr ? r.history + b * r.history_stride : nullptr;
          int len = 0, prompt = 0;
          if (hist != nullptr) {
            len = __ldg(r.history_len + b);
            prompt = r.prompt_len != nullptr ? __ldg(r.prompt_len + b) : 0;
            if ((len < 0 || len > r.max_len) && tid == 0) record(DFLASH2_ERR_INVALID_ARG);
            len = min(max(len, 0), r.max_len);
          }
          __syncthreads();  // (the segment before is done with these)
          for (int i = tid; i < kPickSlice / 32; i += kPickThreads) s.bits[i] = 0u;
          __syncthreads();
          auto mark = [&](int t) {
            const int u = t - lo;
            if (t >= 0 && t < r.V) {
              if (u >= 0 && u < wlen) atomicOr(&s.bits[u >> 5], 1u << (u & 31));
            } else {
              record(DFLASH2_ERR_BAD_INDEX);
            }
          };
          for (int i = tid; i < len; i += kPickThreads) mark(__ldg(hist + i));
          if (r.tokens != nullptr && tid < kTreeRows) {
            uint64_t any = 0;
            for (int i = seg0; i < i1; ++i) any |= s.line[i];
            if ((any >> tid) & 1) mark(__ldg(r.tokens + first + tid));
          }
          for (int e = tid; e < r.n_bias; e += kPickThreads) {
            const int t = __ldg(r.bias_ids + static_cast<int64_t>(b) * r.n_bias + e);
            if (t >= 0) mark(t);
          }
          __syncthreads();
          const uint32_t w0 = s.bits[2 * tid], w1 = s.bits[2 * tid + 1];
          const int mine = __popc(w0) + __popc(w1);
          int inc = mine;
#pragma unroll
          for (int m = 1; m < 32; m <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, m);
            if (lane >= m) inc += v;
          }
          if (lane == 31) s.warp_sum[warp] = inc;
          __syncthreads();
          int at = inc - mine;
          for (int w = 0; w < kPickWarps; ++w) {
            if (w < warp) at += s.warp_sum[w];
            n += s.warp_sum[w];
          }
          s.base[2 * tid] = static_cast<uint16_t>(at);
          s.base[2 * tid + 1] = static_cast<uint16_t>(at + __popc(w0));
#pragma unroll
          for (int h = 0; h < 2; ++h)
            for (uint32_t w = h == 0 ? w0 : w1; w != 0u; w &= w - 1u) {
              offs[at] = static_cast<uint16_t>((2 * tid + h) * 32 + __ffs(w) - 1);
              words[at++] = 0u;
            }
          __syncthreads();
          for (int e = tid; e < r.n_bias; e += kPickThreads) {
            const int u = __ldg(r.bias_ids + static_cast<int64_t>(b) * r.n_bias + e) - lo;
            if (u >= 0 && u < wlen) atomicMax(&words[rank_of(u)], static_cast<uint32_t>(r.n_bias - e) << kBiasShift);
          }
          __syncthreads();
          for (int i = tid; i < len; i += kPickThreads) {
            const int u = __ldg(hist + i) - lo;
            if (u < 0 || u >= wlen) continue;
            if (i < prompt)
              atomicOr(&words[rank_of(u)], kInPrompt);
            else
              atomicAdd(&words[rank_of(u)], 1u);
          }
        }
        const float rep = r.repetition != nullptr ? __ldg(r.repetition + b) : 1.f;
        const float freq = r.frequency != nullptr ? __ldg(r.frequency + b) : 0.f;
        const float pres = r.presence != nullptr ? __ldg(r.presence + b) : 0.f;

        for (int i = seg0; i < i1; ++i) {
          if (s.state[i] != 1) continue;
          const int64_t m = c0 + i;
          const T* row = static_cast<const T*>(r.logits) + m * r.stride + lo;
          T* out = r.out != nullptr ? static_cast<T*>(r.out) + m * r.out_stride + lo : nullptr;
          const uint32_t* allowed = r.mask != nullptr ? reinterpret_cast<const uint32_t*>(r.mask) + m * r.mask_stride + (lo >> 5) : nullptr;
          const bool wide = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
          const bool out_wide = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
          uint4 v[kGroups];
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const int e = (g * kPickThreads + tid) * kN;
            if (wide && e + kN <= wlen)
              v[g] = *reinterpret_cast<const uint4*>(row + e);  // (not by the read-only path: out may be the same buffer)
            else
              v[g] = Vec::load_some(row + e, wlen - e);
          }
          // the drafted ancestors' tokens count for this row
          const uint64_t line = r.tokens != nullptr ? s.line[i] : 0ull;
          auto count_line = [&](uint32_t d) {
            if (tid < kTreeRows && ((line >> tid) & 1)) {
              const int u = __ldg(r.tokens + first + tid) - lo;
              if (u >= 0 && u < wlen) atomicAdd(&words[rank_of(u)], d);
            }
          };
          count_line(1u);
          int* count = &s.count[turn ^= 1];  // (the one before may still be read)
          if (tid == 0) *count = 0;
          __syncthreads();
          float top = -INFINITY;
          for (int k = tid; k < n; k += kPickThreads) {
            const int u = offs[k];
            const uint32_t w = words[k];
            const uint32_t times = w & kCountMask;
            float y = Vec::load(row + u);
            if ((w & (kCountMask | kInPrompt)) != 0u) y = y > 0.f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
            if (times != 0u) y = __fsub_rn(y, __fadd_rn(__fmul_rn(freq, static_cast<float>(times)), pres));
            if ((w >> kBiasShift) != 0u)
              y = __fadd_rn(y, __ldg(r.bias + static_cast<int64_t>(b) * r.n_bias + (r.n_bias - static_cast<int>(w >> kBiasShift))));
            if (allowed != nullptr && !((__ldg(allowed + (u >> 5)) >> (u & 31)) & 1u)) y = -INFINITY;
            vals[k] = y;
            top = max_nan(top, y);
          }
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const int e = (g * kPickThreads + tid) * kN;
            if (e >= wlen) continue;
            if (allowed != nullptr) Vec::drop(v[g], ~(__ldg(allowed + (e >> 5)) >> (e & 31)) & kAll);
            if (out != nullptr) {
              if (out_wide && e + kN <= wlen)
                *reinterpret_cast<uint4*>(out + e) = v[g];
              else
                Vec::store_some(out + e, v[g], wlen - e);
            }
            if (n > 0) Vec::drop(v[g], (s.bits[e >> 5] >> (e & 31)) & kAll);
            top = max_nan(top, Vec::max(v[g]));
          }
          const uint32_t key = pick_key(top);
          const uint32_t most = __reduce_max_sync(lane < 16 ? 0x0000ffffu : 0xffff0000u, key);
          if ((lane & 15) == 0) s.group_max[tid >> 4] = most;
          __syncthreads();
          count_line(~0u);
          if (out != nullptr)
            for (int k = tid; k < n; k += kPickThreads) Vec::store(out + offs[k], vals[k]);
          if (r.K == 0) continue;
          // the K-th largest of the groups' maxima
          const uint32_t g = s.group_max[lane & 15];
          int above = 0;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t o = __shfl_sync(0xffffffffu, g, j);
            above += o > g || (o == g && j < (lane & 15)) ? 1 : 0;
          }
          const uint32_t holder = __ballot_sync(0xffffffffu, above == r.K - 1);
          const uint32_t bound_key = __shfl_sync(0xffffffffu, g, __ffs(holder) - 1);
          const float bound = pick_value(bound_key);
          const unsigned long long prior = sub > 0 && tid < r.K ? s.best[i][tid] : 0ull;
          auto list = [&](unsigned long long entry) {
            const int at = atomicAdd(count, 1);
            if (at < kPickList) s.list[at] = entry;
          };
          auto reaches = [&](float x) { return !(x < bound) && x != -INFINITY; };
          if (prior != 0ull) list(prior);
          for (int k = tid; k < n; k += kPickThreads)
            if (reaches(vals[k])) list(pick_entry(vals[k], lo + offs[k]));
#pragma unroll
          for (int q = 0; q < kGroups; ++q) {
            if (!reaches(Vec::max(v[q]))) continue;
            const int e = (q * kPickThreads + tid) * kN;
#pragma unroll
            for (int j = 0; j < kN; ++j)
              if (reaches(Vec::get(v[q], j))) list(pick_entry(Vec::get(v[q], j), lo + e + j));
          }
          __syncthreads();
          const int listed = *count;
          if (listed <= kPickList) {
            for (int x = tid; x < listed; x += kPickThreads) {
              const unsigned long long mine = s.list[x];
              int before = 0;
              for (int y = 0; y < listed; ++y) before += s.list[y] > mine ? 1 : 0;
              if (before < r.K) s.best[i][before] = mine;
            }
            if (tid < r.K && tid >= listed) s.best[i][tid] = 0ull;
          } else {
            unsigned long long last = ~0ull;
            for (int k = 0; k < r.K; ++k) {
              unsigned long long mine = prior < last ? prior : 0ull;
              auto look = [&](float x, int token) {
                if (x == -INFINITY) return;
                const unsigned long long entry = pick_entry(x, token);
                if (entry < last) mine = max_u64(mine, entry);
              };
              for (int x = tid; x < n; x += kPickThreads) look(vals[x], lo + offs[x]);
#pragma unroll
              for (int q = 0; q < kGroups; ++q) {
                const int e = (q * kPickThreads + tid) * kN;
#pragma unroll
                for (int j = 0; j < kN; ++j) look(Vec::get(v[q], j), lo + e + j);
              }
              mine = warp_max_u64(mine);
              __syncthreads();
              if (lane == 0) s.red[warp] = mine;
              __syncthreads();
              unsigned long long all = 0ull;
              for (int w = 0; w < kPickWarps; ++w) all = max_u64(all, s.red[w]);
              if (tid == 0) s.best[i][k] = all;
              last = all;  // (0, when nothing is left: then nothing is below it)
            }
          }
        }
      }
    }
    if (r.K > 0) {
      // ---- the cluster's lists of each row, merged by one warp
      cluster_sync_all();
      for (int i = rank + a.cluster * warp; i < rows; i += a.cluster * kPickWarps) {
        if (s.state[i] == 0) continue;
        const int64_t m = c0 + i;
        int token = -1;
        float value = -INFINITY;
        if (s.state[i] == 1) {
          unsigned long long mine[8];  // 16 lists of 16 entries at most
          const uint32_t at = smem_u32(&s.best[i][lane & 15]);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int from = 2 * q + (lane >> 4);
            mine[q] = from < a.cluster && (lane & 15) < r.K ? ld_cluster_u64(mapa_shared(at, static_cast<uint32_t>(from))) : 0ull;
          }
          int found = 0;
          for (; found < r.K; ++found) {
            unsigned long long top = 0ull;
#pragma unroll
            for (int q = 0; q < 8; ++q) top = max_u64(top, mine[q]);
            top = warp_max_u64(top);
            if (top == 0ull) break;
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (mine[q] == top) mine[q] = 0ull;
            if (lane == found) {
              token = static_cast<int>(~static_cast<uint32_t>(top));
              value = pick_value(static_cast<uint32_t>(top >> 32));
            }
          }
          // fewer than K tokens above -inf: all of them are here, and the lowest others follow
          for (int t = 0; found < r.K; ++t)
            if (__ballot_sync(0xffffffffu, token == t) == 0u) {
              if (lane == found) token = t;
              ++found;
            }
        }
        if (lane < r.K) {
          r.cand[m * r.K + lane] = token;
          r.unary[m * r.K + lane] = value;
        }
      }
      cluster_sync_all();  // (before the lists are written again, and before a CTA leaves)
    }
  }
}

struct PickPlan {
  int cluster, slice, subs, cap, clusters;
  size_t smem;
};
PickPlan pick_plan(const LogitsTopk& r, int sms) {
  PickPlan p;
  auto slice_of = [&](int cluster, int subs) {
    const int n = cluster * subs;
    return (((r.V + n - 1) / n) + 127) / 128 * 128;
  };
  p.cluster = 1;
  while (p.cluster < 16 && static_cast<int64_t>(p.cluster) * kPickSlice < r.V) p.cluster *= 2;
  // few rows: more CTAs a row, down to 1024 tokens each
  while (p.cluster < 16 && static_cast<int64_t>(r.M) * p.cluster < 2 * sms && r.V / (2 * p.cluster) >= 1024) p.cluster *= 2;
  p.subs = static_cast<int>((r.V + static_cast<int64_t>(p.cluster) * kPickSlice - 1) / (static_cast<int64_t>(p.cluster) * kPickSlice));
  p.slice = slice_of(p.cluster, p.subs);
  const bool named = r.history != nullptr || r.tokens != nullptr || r.n_bias > 0;
  const int most = (r.history != nullptr ? r.max_len : 0) + (r.tokens != nullptr ? kTreeRows : 0) + r.n_bias;
  p.cap = named ? (std::min(p.slice, most) + 7) / 8 * 8 : 0;
  p.smem = static_cast<size_t>(p.cap) * 10;
  // as many clusters as fit at once, each a range of rows
  const int per_sm = std::max(1, std::min(2, static_cast<int>(227 * 1024 / (sizeof(PickShared) + p.smem + 1024))));
  p.clusters = std::max(1, std::min(r.M, sms * per_sm / p.cluster));
  return p;
}

template <typename T>
int launch_pick_t(const PickArgs& a, const PickPlan& p, cudaStream_t st) {
  constexpr int kMost = 10 * kPickSlice;
  static_assert(kMost + sizeof(PickShared) <= 232448, "shared memory");
  static unsigned done = 0, wide = 0;
  auto kern = logits_topk_kernel<T>;
  if (!ensure_smem_attr(kern, kMost, &done)) return fail(DFLASH2_ERR_CUDA, "cudaFuncSetAttribute failed (logits)");
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(DFLASH2_ERR_CUDA, "no device");
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(wide & (1u << (dev & 31)))) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return fail(DFLASH2_ERR_CUDA, "cudaFuncSetAttribute failed (logits)");
      wide |= 1u << (dev & 31);
    }
  }
  cudaLaunchAttribute cl{};
  cl.id = cudaLaunchAttributeClusterDimension;
  cl.val.clusterDim.x = static_cast<unsigned>(p.cluster);
  cl.val.clusterDim.y = 1;
  cl.val.clusterDim.z = 1;
  const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(p.cluster * p.clusters)), dim3(kPickThreads), p.smem, st, &cl, 1, a);
  return e == cudaSuccess ? DFLASH2_OK : fail(DFLASH2_ERR_CUDA, "logits launch failed: %s", cudaGetErrorString(e));
}

}  // namespace

int launch_logits_topk(const LogitsTopk& r, cudaStream_t st) {
  const PickPlan p = pick_plan(r, sm_count());
  PickArgs a{};
  a.r = r;
  a.cluster = p.cluster; a.slice = p.slice; a.subs = p.subs; a.cap = p.cap;
  a.err = device_error_word();
  if (a.err == nullptr) return fail(DFLASH2_ERR_CUDA, "no device error word");
  return r.dtype == DFLASH2_F32 ? launch_pick_t<float>(a, p, st) : launch_pick_t<__nv_bfloat16>(a, p, st);
}

}  // namespace dfl
