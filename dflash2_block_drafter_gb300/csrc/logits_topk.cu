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
// The work is one read of the logits, and what applies to few tokens does not burden the rest. Two kernels:
//  1. Most CTAs stream: every warp reads tiles of 1024 tokens of a row, 32 a lane, and writes one key a lane, the largest
//     value of its allowed tokens. No barriers, nothing shared; the mask is applied to `out` on the way. Between them
//     some CTAs collect what requests name, a CTA a request (and 262144 tokens): the tokens of its history, drafted
//     rows and biases, as a bit a token and as a list of (token, counter), a token's rank among the set bits being its
//     place there; and the rows' requests and lines of ancestors.
//  2. A CTA a row selects. The named tokens' values are computed, and the lanes that hold a named token marked, whose
//     keys say too much. The other keys (a 32nd of the row) and the named values give a bound that the K best reach:
//     the K-th largest of 32 groups' maxima. The few lanes whose key reaches it are read once more, and the K best of
//     what reaches the bound there, and of the named, are ranked by (value, lower token). Where more reach it than can be
//     ranked (equal values; strong penalties for a history that names nearly every lane), the best of each of 1024
//     shares of them give a nearer bound, for two passes more; a row of which up to four tokens are wanted, or whose tokens
//     fall into few shares, is searched in K rounds instead. (63 rows of 32771 with 30000 generated tokens, K = 16: 47 us
//     under penalties of 1.1, 0.1 and 0.1, 92 under 1.5, 1 and 1; in K rounds 222.)
// What bounds it: 64 x 15 rows of 248320 fp32 tokens take 168 us, 0.85 of the copy rate; 64 bf16 rows under masks, adjusted
// logits wanted, 30 us (25 where logits and out stay in L2 from call to call); one block's 15 rows 14.9 us and rows with
// histories of 30000 tokens 50: the latency of two launches and, of the names, of a history's atomics, their ranks and the
// named tokens' values. (In the rules below each pair of figures was measured side by side.)
// (One kernel that kept a row's slices in the registers or shared memory of a cluster took 792 us for the first:
// barriers, and 27 instructions a token.)
//
// Only what is above -inf is a candidate; rows with fewer than K such tokens are filled with the lowest of the others.
#include <algorithm>

#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"
#include "tree.cuh"
#include "warp_keys.cuh"

namespace dfl {
namespace {

constexpr int kWindowLog = 18, kWindow = 1 << kWindowLog;  // tokens whose names a CTA collects
constexpr int kTile = 1024;                                // tokens a warp reads at a time,
constexpr int kLaneTokens = 32;                            // of which a lane has
constexpr int kStreamThreads = 512, kStreamWarps = kStreamThreads / 32;
constexpr int kStreamTiles = 4;                            // tiles a warp, at most
constexpr int kEntries = 1024, kLanes = 512;               // that reach the bound
constexpr int kFewWanted = 4;                              // K up to which a row where more reach it is searched at once
constexpr int kPickK = 16;
constexpr uint32_t kCountMask = (1u << 20) - 1, kInPrompt = 1u << 20;  // a counter; over it, which bias
constexpr int kBiasShift = 21;
constexpr uint32_t kDrafted = 1u << 31;  // beside a named token: one of the request's drafted rows has it

struct PickArgs {
  LogitsTopk r;
  int each;             // rows a request, 0: as row_off says
  int windows, cap;     // windows of the vocabulary (0: nothing is named); counters a window
  int words;            // of bits a request
  int tiles;            // a row
  int warp_tiles, row_warps, stream_ctas, other_ctas;  // of the first kernel
  int counters, kept;   // named tokens' counters and values that shared memory holds, at most
  uint32_t* bits;       // [B][words]
  int* named;           // [B][windows] how many
  uint2* names;         // [B][windows][cap] (token, counter)
  int* request;         // [M] each row's, -1: none (row_off given)
  uint64_t* line;       // [M] the row's drafted ancestors, 0: it is not there (tokens given)
  uint32_t* keys;       // [M][tiles][32]
  int* err;
};

__device__ __forceinline__ void record(int* err, int status) { atomicCAS(err, 0, status); }

// An order-preserving key; NaN above every number (and an entry of it below all ones).
constexpr uint32_t kKeyNan = 0xfffffffeu;
__device__ __forceinline__ uint32_t pick_key(float v) { return v != v ? kKeyNan : float_key(v); }
__device__ __forceinline__ float pick_value(uint32_t k) { return k == kKeyNan ? __uint_as_float(0x7fffffffu) : key_float(k); }
__device__ __forceinline__ unsigned long long pick_entry(float v, int token) {
  return (static_cast<unsigned long long>(pick_key(v)) << 32) | static_cast<uint32_t>(~token);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ unsigned long long max_u64(unsigned long long a, unsigned long long b) { return a > b ? a : b; }
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<unsigned long long>(hi) << 32) | lo;
}

// ------------------------------------------------------------------ names
// The history's tokens and their places, four of them a load and four loads in flight.
template <typename F>
__device__ __forceinline__ void for_history(const int32_t* hist, int len, F f) {
  const int tid = static_cast<int>(threadIdx.x);
  const int head = min(len, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(hist) & 15u)) & 15u) / 4);
  const int quads = (len - head) / 4, tail = head + 4 * quads;
  if (tid < head) f(__ldg(hist + tid), tid);
  if (tid < len - tail) f(__ldg(hist + tail + tid), tail + tid);
  const int4* wide = reinterpret_cast<const int4*>(hist + head);
  for (int i = tid; i < quads; i += 4 * kStreamThreads) {
    int4 q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * kStreamThreads < quads) q[k] = __ldg(wide + i + k * kStreamThreads);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k * kStreamThreads >= quads) break;
      const int at = head + 4 * (i + k * kStreamThreads);
      f(q[k].x, at);
      f(q[k].y, at + 1);
      f(q[k].z, at + 2);
      f(q[k].w, at + 3);
    }
  }
}

// The request of row m in [0, M), by a binary search: the last that starts at or before it, if its span holds it (and
// the row is among its first 64 where they are drafted); else -1.
__device__ __forceinline__ int ragged_request(const LogitsTopk& r, int m, bool& late) {
  int lo = 0, hi = r.B - 1;
  // (ordinary loads: the spans may be what a page plan in front has just written)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (r.row_off[mid] <= m)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int first = r.row_off[lo];
  const bool in = first >= 0 && first <= m && m < r.row_off[lo + 1];
  late = in && r.tokens != nullptr && m - first >= kTreeRows;
  return in && !late ? lo : -1;
}
// A warp's work: the lines of a request's first 64 rows, from row `first` on.
__device__ __forceinline__ TreeLines request_lines(const PickArgs& a, int b, int& first, int& rows, bool& bad) {
  const LogitsTopk& r = a.r;
  const int lane = static_cast<int>(threadIdx.x) & 31;
  rows = a.each;
  first = b * a.each;
  if (a.each == 0) {
    first = r.row_off[b];
    rows = first < 0 ? 0 : min(r.row_off[b + 1], r.M) - first;
  }
  rows = min(rows, kTreeRows);
  int parent[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = lane + 32 * h;
    parent[h] = t < rows ? (r.parents != nullptr ? __ldg(r.parents + first + t) : t - 1) : -2;
  }
  return tree_lines(parent, rows, bad);
}

// The requests of rows x 512 .. (row_off given), and the check of the spans.
__device__ __forceinline__ void map_rows(const PickArgs& a, int x, int ctas) {
  const LogitsTopk& r = a.r;
  const int m = x * kStreamThreads + static_cast<int>(threadIdx.x);
  for (int b = m; b < r.B; b += ctas * kStreamThreads) {
    const int lo = r.row_off[b], hi = r.row_off[b + 1];
    if (lo < 0 || hi < lo || hi > r.M) record(a.err, DFLASH2_ERR_INVALID_ARG);
  }
  if (m >= r.M) return;
  bool late;
  a.request[m] = ragged_request(r, m, late);
  if (late) record(a.err, DFLASH2_ERR_INVALID_ARG);
}

// What request b names in a window. Shared memory: bits, four words of which share a base, their first's rank.
__device__ __forceinline__ void collect_names(const PickArgs& a, int x, uint32_t* bits) {
  const LogitsTopk& r = a.r;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int b = x / a.windows, window = x - b * a.windows;
  const int lo = window << kWindowLog, len = min(kWindow, r.V - lo);
  const int quads = (len + 127) / 128;                         // of words of bits
  uint32_t* base = bits + quads * 4;                           // [quads]
  __shared__ int warp_sum[kStreamWarps];
  __shared__ uint64_t there;                                   // the request's drafted rows that are there
  const int32_t* hist = nullptr;
  int hist_len = 0, prompt = 0;
  if (r.history != nullptr) {
    hist = r.history + b * r.history_stride;
    hist_len = __ldg(r.history_len + b);
    prompt = r.prompt_len != nullptr ? __ldg(r.prompt_len + b) : 0;
    if ((hist_len < 0 || hist_len > r.max_len) && tid == 0) record(a.err, DFLASH2_ERR_INVALID_ARG);
    hist_len = min(max(hist_len, 0), r.max_len);
  }
  uint4* bits4 = reinterpret_cast<uint4*>(bits);
  for (int k = tid; k < quads; k += kStreamThreads) bits4[k] = make_uint4(0u, 0u, 0u, 0u);
  int first = 0;
  if (r.tokens != nullptr && warp == 0) {
    int rows;
    bool bad;
    const TreeLines tree = request_lines(a, b, first, rows, bad);
    if (bad) record(a.err, DFLASH2_ERR_BAD_INDEX);
    const uint32_t in0 = __ballot_sync(0xffffffffu, tree.line[0] != 0ull), in1 = __ballot_sync(0xffffffffu, tree.line[1] != 0ull);
    if (lane == 0) there = (static_cast<uint64_t>(in1) << 32) | in0;
    if (window == 0)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < rows) a.line[first + lane + 32 * h] = tree.line[h];
  }
  __syncthreads();
  auto mark = [&](int t) {
    const int u = t - lo;
    if (t >= 0 && t < r.V) {
      // (most of a history repeats)
      if (u >= 0 && u < len && !((bits[u >> 5] >> (u & 31)) & 1u)) atomicOr(&bits[u >> 5], 1u << (u & 31));
    } else {
      record(a.err, DFLASH2_ERR_BAD_INDEX);
    }
  };
  const int32_t* bias_ids = r.bias_ids + static_cast<int64_t>(b) * r.n_bias;
  for_history(hist, hist_len, [&](int t, int) { mark(t); });
  if (r.tokens != nullptr && warp == 0)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if ((there >> (lane + 32 * h)) & 1) mark(__ldg(r.tokens + first + lane + 32 * h));
  for (int e = tid; e < r.n_bias; e += kStreamThreads) {
    const int t = __ldg(bias_ids + e);
    if (t >= 0) mark(t);
  }
  __syncthreads();
  // ranks: a warp has a range of the quads, 32 at a time
  const int span = (quads + kStreamWarps - 1) / kStreamWarps, q0 = min(quads, warp * span), q1 = min(quads, q0 + span);
  auto ones = [](const uint4& w) { return __popc(w.x) + __popc(w.y) + __popc(w.z) + __popc(w.w); };
  int sum = 0;
  for (int q = q0 + lane; q < q1; q += 32) sum += ones(bits4[q]);
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) warp_sum[warp] = sum;
  __syncthreads();
  int at = 0, n = 0;
#pragma unroll
  for (int w = 0; w < kStreamWarps; ++w) {
    if (w < warp) at += warp_sum[w];
    n += warp_sum[w];
  }
  if (tid == 0) a.named[b * a.windows + window] = n;
  uint2* names = a.names + static_cast<int64_t>(b * a.windows + window) * a.cap;
  uint32_t* to = a.bits + static_cast<int64_t>(b) * a.words + (lo >> 5);
  for (int qq = q0; qq < q1; qq += 32) {
    const int q = qq + lane;
    const uint4 w = q < q1 ? bits4[q] : make_uint4(0u, 0u, 0u, 0u);
    const int mine = ones(w);
    int inc = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, m);
      if (lane >= m) inc += v;
    }
    if (q < q1) base[q] = static_cast<uint32_t>(at + inc - mine);
    at += __shfl_sync(0xffffffffu, inc, 31);
  }
  for (int w = tid; w < (len + 31) / 32; w += kStreamThreads) to[w] = bits[w];
  if (n == 0) return;
  // counters of 16 bits, and a bit for the prompt's, beside the bits if they fit there (an SM's atomics on global memory
  // go at one a clock, and on one address far slower)
  uint32_t* counts = a.counters > 0 ? base + quads : nullptr;  // [counters / 2]
  uint32_t* in_prompt = counts + a.counters / 2;               // [counters / 32]
  for (int k = tid; k < n; k += kStreamThreads) names[k].y = 0u;
  for (int k = tid; k < (a.counters > 0 ? n / 2 + 1 : 0); k += kStreamThreads) counts[k] = 0u;
  for (int k = tid; k < (a.counters > 0 ? n / 32 + 1 : 0); k += kStreamThreads) in_prompt[k] = 0u;
  __syncthreads();
  // (a token that is named more than once writes its name more than once, the same each time)
  auto place_name = [&](int t) {
    const int u = t - lo;
    if (t < 0 || u < 0 || u >= len) return -1;
    const int i = (u >> 5) & 3;
    const uint4 w = bits4[u >> 7];
    const uint32_t below = (1u << (u & 31)) - 1u;
    const int k = static_cast<int>(base[u >> 7]) + __popc(w.x & (i > 0 ? ~0u : below)) + (i > 0 ? __popc(w.y & (i > 1 ? ~0u : below)) : 0) +
                  (i > 1 ? __popc(w.z & (i > 2 ? ~0u : below)) : 0) + (i > 2 ? __popc(w.w & below) : 0);
    names[k].x = static_cast<uint32_t>(t);
    return k;
  };
  if (r.n_bias > 0) {
    for (int e = tid; e < r.n_bias; e += kStreamThreads) {
      const int k = place_name(__ldg(bias_ids + e));
      if (k >= 0) atomicMax(&names[k].y, static_cast<uint32_t>(r.n_bias - e) << kBiasShift);
    }
    __syncthreads();
  }
  for_history(hist, hist_len, [&](int t, int at_place) {
    const int k = place_name(t);
    if (k < 0) return;
    if (counts == nullptr)
      at_place < prompt ? atomicOr(&names[k].y, kInPrompt) : atomicAdd(&names[k].y, 1u);
    else if (at_place < prompt)
      atomicOr(in_prompt + (k >> 5), 1u << (k & 31));
    else
      atomicAdd(counts + (k >> 1), 1u << (16 * (k & 1)));
  });
  __syncthreads();
  if (counts != nullptr)
    for (int k = tid; k < n; k += kStreamThreads)
      names[k].y += ((counts[k >> 1] >> (16 * (k & 1))) & 0xffffu) + (((in_prompt[k >> 5] >> (k & 31)) & 1u) != 0u ? kInPrompt : 0u);
  if (r.tokens != nullptr && warp == 0)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if ((there >> (lane + 32 * h)) & 1) {
        const int t = __ldg(r.tokens + first + lane + 32 * h), k = place_name(t);
        if (k >= 0) names[k].x = static_cast<uint32_t>(t) | kDrafted;
      }
}

// ------------------------------------------------------------------ stream
// Sixteen bytes of logits. (No loads by the read-only path: `out` may be the same buffer.)
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}
// Four bits as the top bits of four bytes, whose signs are then spread over the bytes of elements.
__device__ __forceinline__ uint32_t spread4(uint32_t bits) { return (bits & 15u) * 0x10204080u; }
template <uint32_t kSelect>
__device__ __forceinline__ uint32_t signs(uint32_t x) {  // (8 + i: the sign of byte i)
  uint32_t y;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(y) : "r"(x), "n"(kSelect));
  return y;
}
__device__ __forceinline__ uint32_t choose(uint32_t mask, uint32_t a, uint32_t b) { return (a & mask) | (b & ~mask); }
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
    const uint32_t x = spread4(bits);
    u.x = choose(signs<0x8888>(x), 0xff800000u, u.x);
    u.y = choose(signs<0x9999>(x), 0xff800000u, u.y);
    u.z = choose(signs<0xaaaa>(x), 0xff800000u, u.z);
    u.w = choose(signs<0xbbbb>(x), 0xff800000u, u.w);
  }
  static __device__ __forceinline__ float max(float m, const uint4& u) {
    return max3_nan(max3_nan(m, __uint_as_float(u.x), __uint_as_float(u.y)), __uint_as_float(u.z), __uint_as_float(u.w));
  }
  // elements [from, to) of them; the others are -inf
  static __device__ __forceinline__ uint4 load_some(const float* p, int from, int to) {
    uint4 u;
    u.x = from <= 0 && to > 0 ? __float_as_uint(p[0]) : 0xff800000u;
    u.y = from <= 1 && to > 1 ? __float_as_uint(p[1]) : 0xff800000u;
    u.z = from <= 2 && to > 2 ? __float_as_uint(p[2]) : 0xff800000u;
    u.w = from <= 3 && to > 3 ? __float_as_uint(p[3]) : 0xff800000u;
    return u;
  }
  static __device__ __forceinline__ void store_some(float* p, const uint4& u, int from, int to) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j >= from && j < to) p[j] = get(u, j);
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
  static __device__ __forceinline__ void drop(uint4& u, uint32_t bits) {
    const uint32_t x = spread4(bits), y = spread4(bits >> 4);
    u.x = choose(signs<0x9988>(x), 0xff80ff80u, u.x);
    u.y = choose(signs<0xbbaa>(x), 0xff80ff80u, u.y);
    u.z = choose(signs<0x9988>(y), 0xff80ff80u, u.z);
    u.w = choose(signs<0xbbaa>(y), 0xff80ff80u, u.w);
  }
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  static __device__ __forceinline__ float max(float m, const uint4& u) {
    const __nv_bfloat162 x = __hmax2_nan(__hmax2_nan(two(u.x), two(u.y)), __hmax2_nan(two(u.z), two(u.w)));
    return max3_nan(m, __low2float(x), __high2float(x));
  }
  static __device__ __forceinline__ uint4 load_some(const __nv_bfloat16* p, int from, int to) {
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i >= from && 2 * i < to ? q[2 * i] : 0xff80u;
      const uint32_t hi = 2 * i + 1 >= from && 2 * i + 1 < to ? q[2 * i + 1] : 0xff80u;
      w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void store_some(__nv_bfloat16* p, const uint4& u, int from, int to) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= from && j < to) reinterpret_cast<unsigned short*>(p)[j] = static_cast<unsigned short>(word(u, j >> 1) >> (16 * (j & 1)));
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};

// A row: its request (-1: it belongs to none, or is not there), and its first element's place in sixteen bytes: the
// tiles lie on sixteen-byte boundaries, tile x's lane l has tokens x 1024 + g 32 n + l n - off + (0 .. n - 1).
struct PickRow {
  int request, first;
  bool missing;  // a drafted row that is not there
};
__device__ __forceinline__ PickRow pick_row(const PickArgs& a, int m) {
  PickRow p;
  p.request = a.each > 0 ? m / a.each : a.request[m];
  p.first = a.each > 0 ? p.request * a.each : (p.request >= 0 ? a.r.row_off[p.request] : 0);
  p.missing = p.request >= 0 && a.r.tokens != nullptr && a.line[m] == 0ull;
  return p;
}
template <typename T>
__device__ __forceinline__ int row_offset(const T* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}
// Bits t .. t + 31 of a row of `words` words (0 outside them); t may be negative, by less than 32.
__device__ __forceinline__ uint32_t bits_from(const uint32_t* w, int words, int t) {
  const int i = t >> 5;
  const uint32_t lo = i >= 0 && i < words ? __ldg(w + i) : 0u;
  if ((t & 31) == 0) return lo;
  return __funnelshift_r(lo, i + 1 < words ? __ldg(w + i + 1) : 0u, t & 31);
}

template <typename T>
__device__ __forceinline__ void stream_row(const PickArgs& a, int x) {
  using Vec = PickVec<T>;
  constexpr int kN = Vec::kN, kG = kLaneTokens / kN;
  const LogitsTopk& r = a.r;
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const int at = x * kStreamWarps + warp, m = at / a.row_warps;  // (rows side by side: short ones leave no warp idle)
  if (m >= r.M) return;
  const int tile0 = (at - m * a.row_warps) * a.warp_tiles;
  const T* row = static_cast<const T*>(r.logits) + static_cast<int64_t>(m) * r.stride;
  T* out = r.out != nullptr ? static_cast<T*>(r.out) + static_cast<int64_t>(m) * r.out_stride : nullptr;
  const int off = row_offset(row), mask_words = (r.V + 31) / 32;
  const bool out_wide = out != nullptr && row_offset(out) == off;
  const uint32_t* mask = r.mask != nullptr ? reinterpret_cast<const uint32_t*>(r.mask) + static_cast<int64_t>(m) * r.mask_stride : nullptr;
  if (out != nullptr && (a.each == 0 || r.tokens != nullptr)) {
    // rows of no request, and drafted rows that are not there, keep what `out` holds
    bool late, bad;
    int first, rows;
    const int b = a.each > 0 ? m / a.each : ragged_request(r, m, late);
    if (b < 0) return;
    if (r.tokens != nullptr) {
      const TreeLines tree = request_lines(a, b, first, rows, bad);
      if (!__any_sync(0xffffffffu, (m - first == lane && tree.line[0] != 0ull) || (m - first == lane + 32 && tree.line[1] != 0ull)))
        return;
    }
  }
  for (int tile = tile0; tile < min(tile0 + a.warp_tiles, a.tiles); ++tile) {
    const int t0 = tile * kTile - off;  // the tile's first token
    const bool inside = t0 >= 0 && t0 + kTile <= r.V;
    uint4 v[kG];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int t = t0 + (g * 32 + lane) * kN;
      if (inside || (t >= 0 && t + kN <= r.V))
        v[g] = load16(row + t);
      else
        v[g] = Vec::load_some(row + t, -t, r.V - t);
    }
    if (mask != nullptr) {
      const uint32_t denied = ~bits_from(mask, mask_words, t0 + 32 * lane);  // lane l holds bits 32 l .. of the tile
      if (__any_sync(0xffffffffu, denied != 0u)) {
#pragma unroll
        for (int g = 0; g < kG; ++g)  // those of the lane's g-th sixteen bytes
          Vec::drop(v[g], __shfl_sync(0xffffffffu, denied, (g * 32 + lane) * kN / 32) >> (lane * kN & 31));
      }
    }
    if (out != nullptr)
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        const int t = t0 + (g * 32 + lane) * kN;
        if (out_wide && t >= 0 && t + kN <= r.V)
          *reinterpret_cast<uint4*>(out + t) = v[g];
        else
          Vec::store_some(out + t, v[g], -t, r.V - t);
      }
    if (r.K == 0) continue;
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < kG; ++g) top = Vec::max(top, v[g]);
    a.keys[(static_cast<int64_t>(m) * a.tiles + tile) * 32 + lane] = pick_key(top);
  }
}

// The streaming CTAs, and evenly between them those that collect names and map rows.
template <typename T>
__global__ void __launch_bounds__(kStreamThreads) logits_stream_kernel(const PickArgs a) {
  extern __shared__ __align__(16) uint32_t stream_smem[];
  pdl_trigger();
  pdl_wait();
  const long long x = blockIdx.x, all = gridDim.x;
  const int other = static_cast<int>(x * a.other_ctas / all);
  if (static_cast<int>((x + 1) * a.other_ctas / all) == other) {
    stream_row<T>(a, static_cast<int>(x) - other);
  } else if (other < a.r.B * a.windows) {
    collect_names(a, other, stream_smem);
  } else {
    map_rows(a, other - a.r.B * a.windows, a.other_ctas - a.r.B * a.windows);
  }
}

// ------------------------------------------------------------------ select
// Which of kEntries shares a token falls into, spread by a product's upper bits (multiplicative hashing, Knuth).
__device__ __forceinline__ int share_of(int token) { return static_cast<int>((static_cast<uint32_t>(token) * 0x9e3779b1u) >> 22); }
static_assert(kEntries == 1 << 10, "shares");

struct SelectShared {
  unsigned long long entry[kEntries];
  unsigned long long least;
  unsigned long long best[kPickK];
  unsigned long long red[32];
  int lane[kLanes];
  alignas(16) uint32_t group_max[32];
  int entries, lanes;
};

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads <= 512 ? 1536 / kThreads : 1) logits_select_kernel(const PickArgs a) {
  using Vec = PickVec<T>;
  constexpr int kN = Vec::kN, kWarps = kThreads / 32;
  constexpr int kKeyLoads = kThreads >= 512 ? 2048 / kThreads : 0;  // sixteen bytes of keys a thread keeps
  constexpr int kBatch = kThreads == 1024 ? 4 : 2;                  // named tokens a thread has in flight
  __shared__ SelectShared s;
  extern __shared__ uint32_t marked[];  // [tiles] lanes that hold a named token
  float* kept = reinterpret_cast<float*>(marked + a.tiles);  // [kept] named tokens' values
  const LogitsTopk& r = a.r;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int m = static_cast<int>(blockIdx.x);
  if (tid == 0) s.entries = s.lanes = 0;
  if (tid < kPickK) s.best[tid] = 0ull;
  if (tid < 32) s.group_max[tid] = static_cast<uint32_t>(tid);
  if (r.K > 0)
    for (int k = tid; k < a.tiles; k += kThreads) marked[k] = 0u;
  pdl_trigger();
  pdl_wait();
  const PickRow p = pick_row(a, m);
  if (p.request < 0) return;
  if (p.missing) {
    if (tid < r.K) {
      r.cand[static_cast<int64_t>(m) * r.K + tid] = -1;
      r.unary[static_cast<int64_t>(m) * r.K + tid] = -INFINITY;
    }
    return;
  }
  const int b = p.request;
  const T* row = static_cast<const T*>(r.logits) + static_cast<int64_t>(m) * r.stride;
  T* out = r.out != nullptr ? static_cast<T*>(r.out) + static_cast<int64_t>(m) * r.out_stride : nullptr;
  const int off = row_offset(row), quads = r.K > 0 ? a.tiles * 8 : 0;
  const uint4* keys = reinterpret_cast<const uint4*>(a.keys + static_cast<int64_t>(m) * a.tiles * 32);
  uint4 key[kKeyLoads > 0 ? kKeyLoads : 1];
#pragma unroll
  for (int j = 0; j < kKeyLoads; ++j)
    key[j] = tid + j * kThreads < quads ? keys[tid + j * kThreads] : make_uint4(0u, 0u, 0u, 0u);
  const uint32_t* mask = r.mask != nullptr ? reinterpret_cast<const uint32_t*>(r.mask) + static_cast<int64_t>(m) * r.mask_stride : nullptr;
  const uint32_t* taken = a.windows > 0 ? a.bits + static_cast<int64_t>(b) * a.words : nullptr;
  const float rep = r.repetition != nullptr ? __ldg(r.repetition + b) : 1.f;
  const float freq = r.frequency != nullptr ? __ldg(r.frequency + b) : 0.f;
  const float pres = r.presence != nullptr ? __ldg(r.presence + b) : 0.f;
  // the drafted tokens on the row's line, one or two a lane of every warp
  uint64_t line = 0;
  int drafted[2] = {-1, -1};
  if (r.tokens != nullptr) {
    line = a.line[m] & ((2ull << min(m - p.first, kTreeRows - 1)) - 1ull);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if ((line >> (lane + 32 * h)) & 1) drafted[h] = __ldg(r.tokens + p.first + lane + 32 * h);
  }
  auto bit_of = [](const uint32_t* w, int t) { return (w[t >> 5] >> (t & 31)) & 1u; };
  int named = 0;
  // (what the first kernel writes is read by ordinary loads: this one may have started before it ended)
  for (int w = 0; w < a.windows; ++w) named += a.named[b * a.windows + w];
  auto name_at = [&](int place) {  // of the request's lists, one behind the other
    int w = b * a.windows;
    for (int n; place >= (n = a.named[w]); ++w) place -= n;
    return a.names[static_cast<int64_t>(w) * a.cap + place];
  };
  // f(token, value, place) of the thread's named tokens from place `from` on (a multiple of 32; whole warps)
  auto for_named = [&](int from, auto f) {
    for (int p0 = from + warp * 32; p0 < named; p0 += kBatch * kThreads) {
      uint2 name[kBatch];
      float y[kBatch];
      int token[kBatch];
      uint32_t ok[kBatch];
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        const int place = p0 + h * kThreads + lane;
        name[h] = place < named ? name_at(place) : make_uint2(0xffffffffu, 0u);
      }
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        token[h] = name[h].x != 0xffffffffu ? static_cast<int>(name[h].x & ~kDrafted) : -1;
        ok[h] = token[h] >= 0 && mask != nullptr ? bit_of(mask, token[h]) : 1u;
        y[h] = token[h] >= 0 ? Vec::load(row + token[h]) : 0.f;
      }
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        const int t = token[h];
        uint32_t times = name[h].y & kCountMask;
        if (__any_sync(0xffffffffu, t >= 0 && (name[h].x & kDrafted) != 0u))
          for (uint64_t left = line; left != 0ull; left &= left - 1ull) {
            const int at = __ffsll(static_cast<long long>(left)) - 1;
            if (__shfl_sync(0xffffffffu, at < 32 ? drafted[0] : drafted[1], at & 31) == t) ++times;
          }
        if (t < 0) continue;
        float x = y[h];
        if (times != 0u || (name[h].y & kInPrompt) != 0u) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
        if (times != 0u) x = __fsub_rn(x, __fadd_rn(__fmul_rn(freq, static_cast<float>(times)), pres));
        if ((name[h].y >> kBiasShift) != 0u)
          x = __fadd_rn(x, __ldg(r.bias + static_cast<int64_t>(b) * r.n_bias + (r.n_bias - static_cast<int>(name[h].y >> kBiasShift))));
        f(t, ok[h] != 0u ? x : -INFINITY, p0 + h * kThreads + lane);
      }
    }
  };
  // (out may be the logits themselves: a value that is not kept is stored after the last look)
  float top_named = -INFINITY;
  __syncthreads();
  for_named(0, [&](int t, float y, int place) {
    if (r.K > 0) atomicOr(&marked[(t + off) >> 10], 1u << ((t + off) / kN & 31));
    top_named = max_nan(top_named, y);
    if (place < a.kept) kept[place] = y;
    if (out != nullptr && place < a.kept) Vec::store(out + t, y);
  });
  // once more, those that reach a key
  auto again = [&](uint32_t key, auto f) {
    for (int place = tid; place < min(named, a.kept); place += kThreads)
      if (pick_key(kept[place]) >= key) f(static_cast<int>(name_at(place).x & ~kDrafted), kept[place]);
    for_named(a.kept, [&](int t, float y, int) { f(t, y); });
  };
  auto store_rest = [&]() {
    if (out != nullptr) for_named(a.kept, [&](int t, float y, int) { Vec::store(out + t, y); });
  };
  if (r.K == 0) {
    store_rest();
    return;
  }
  __syncthreads();
  // the largest keys of lanes without a named token, and of any. In 32 groups, by a lane's place in its tile: those of a
  // short row are spread over all of them. (By runs of threads, 1024 tokens were one group, and a row of them
  // entered whole: 4096 rows took 680 us.) Named tokens count by the threads that hold them.
  uint32_t top[4] = {0u, 0u, 0u, 0u}, top_any = 0u;
  auto look_at = [&](int k, const uint4& q) {
    const uint32_t mark = marked[k >> 3] >> (4 * k & 31);
    const uint32_t v[4] = {q.x, q.y, q.z, q.w};
    top_any = max(top_any, max(max(q.x, q.y), max(q.z, q.w)));
#pragma unroll
    for (int j = 0; j < 4; ++j) top[j] = max(top[j], (mark >> j & 1u) != 0u ? 0u : v[j]);
  };
#pragma unroll
  for (int j = 0; j < kKeyLoads; ++j)
    if (tid + j * kThreads < quads) look_at(tid + j * kThreads, key[j]);
#pragma unroll 4
  for (int k = tid + kKeyLoads * kThreads; k < quads; k += kThreads) look_at(k, keys[k]);
  const uint32_t named_key = pick_key(top_named);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t most = (warp & 3) == j ? max(top[j], named_key) : top[j];
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 8));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 16));
    // (the lowest bits tell groups apart: the K-th largest is one of them, and without these bits not above it)
    const uint32_t group = static_cast<uint32_t>(4 * lane + j);
    if (lane < 8) atomicMax(&s.group_max[group], (most & ~31u) | group);
  }
  __syncthreads();
  const uint32_t g = s.group_max[lane];
  int above = 0;
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(&s.group_max[j]);
    above += (o.x > g) + (o.y > g) + (o.z > g) + (o.w > g);
  }
  const uint32_t holder = __ballot_sync(0xffffffffu, above == r.K - 1);
  constexpr uint32_t kMinusInf = 0x007fffffu;  // the key of -inf
  const uint32_t bound = max(__shfl_sync(0xffffffffu, g, __ffs(holder) - 1) & ~31u, kMinusInf + 1u);
  auto list_lanes = [&](int k, const uint4& q) {
    if (max(max(q.x, q.y), max(q.z, q.w)) < bound) return;
    const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (x[j] >= bound) {
        const int at = atomicAdd(&s.lanes, 1);
        if (at < kLanes) s.lane[at] = 4 * k + j;
      }
  };
  if (top_any >= bound) {
#pragma unroll
    for (int j = 0; j < kKeyLoads; ++j) list_lanes(tid + j * kThreads, key[j]);
#pragma unroll 4
    for (int k = tid + kKeyLoads * kThreads; k < quads; k += kThreads) list_lanes(k, keys[k]);
  }
  auto free_value = [&](int t) {  // of a token that is allowed and not named, else -inf
    const uint32_t named = taken != nullptr ? bit_of(taken, t) : 0u, ok = mask != nullptr ? bit_of(mask, t) : 1u;
    const float x = Vec::load(row + t);
    return named == 0u && ok != 0u ? x : -INFINITY;
  };
  // Pass 0: what reaches the bound. Where that is more than can be ranked, pass 1 keeps the best of each of 1024 shares of
  // it, whose K-th largest is a bound that few besides the K best reach, and pass 2 takes those. (A named token's lane counts
  // by the token's own logit, and where a history names nearly all lanes the bound is weak: 63 rows of 32771 under
  // penalties of 1.5, 1 and 1 for 30000 generated tokens list up to 1024 lanes and 7432 values.)
  unsigned long long least = static_cast<unsigned long long>(bound) << 32;
  int n;
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    const uint32_t least_key = static_cast<uint32_t>(least >> 32);
    auto take = [&](float x, int token) {
      const unsigned long long e = pick_entry(x, token);
      if (e < least) return;
      if (pass == 1) {
        unsigned long long* share = &s.entry[share_of(token)];
        if (e > *share) atomicMax(share, e);
        return;
      }
      const int at = atomicAdd(&s.entries, 1);
      if (at < kEntries) s.entry[at] = e;
    };
    if (__any_sync(0xffffffffu, named_key >= least_key)) again(least_key, [&](int t, float y) { take(y, t); });
    __syncthreads();
    auto take_lane = [&](int x) {  // the tokens of the row's lane x, one a lane here
      const int t = (x >> 5) * kTile + ((lane / kN) * 32 + (x & 31)) * kN + lane % kN - off;
      const bool full = *reinterpret_cast<volatile int*>(&s.entries) > kEntries;  // (too many: the rest is not looked at)
      if (t >= 0 && t < r.V && !full) take(free_value(t), t);
    };
    const int lanes = s.lanes;
    if (lanes <= kLanes) {
#pragma unroll 4
      for (int k = warp; k < lanes; k += kWarps) take_lane(s.lane[k]);
    } else {  // more than are listed: the keys once more
      const uint32_t* each = reinterpret_cast<const uint32_t*>(keys);
      for (int x0 = warp * 32; x0 < 4 * quads; x0 += kThreads)
        for (uint32_t hit = __ballot_sync(0xffffffffu, each[x0 + lane] >= least_key); hit != 0u; hit &= hit - 1u)
          take_lane(x0 + __ffs(hit) - 1);
    }
    __syncthreads();
    n = s.entries;
    // (up to four tokens the search below, a pass a token, is as fast: 15 rows of 248320 equal values take 76 us for one, 121
    // for two and 748 for sixteen by it, 200 by shares)
    if (pass == 2 || (pass == 0 && (n <= kEntries || r.K <= kFewWanted))) break;
    __syncthreads();
    if (pass == 0) {
      for (int x = tid; x < kEntries; x += kThreads) s.entry[x] = 0ull;
      if (tid == 0) {
        s.entries = 0;
        s.least = 0ull;
      }
      __syncthreads();
      continue;
    }
    for (int x = tid; x < kEntries; x += kThreads) {
      const unsigned long long mine = s.entry[x];
      int before = 0;
#pragma unroll 4
      for (int y = 0; y < kEntries; ++y) before += s.entry[y] > mine ? 1 : 0;
      if (before == r.K - 1 && mine != 0ull) s.least = mine;
    }
    __syncthreads();
    least = max_u64(least, s.least);  // (fewer than K shares have any: as it was)
  }
  if (n <= kEntries) {
    for (int x = tid; x < n; x += kThreads) {
      const unsigned long long mine = s.entry[x];
      int before = 0;
#pragma unroll 4
      for (int y = 0; y < n; ++y) before += s.entry[y] > mine ? 1 : 0;
      if (before < r.K) s.best[before] = mine;
    }
    __syncthreads();
  } else {  // (few wanted, or tokens of few shares)
    unsigned long long last = ~0ull;
#pragma unroll 1
    for (int k = 0; k < r.K; ++k) {
      unsigned long long mine = 0ull;
      auto look = [&](int t, float x) {
        if (x == -INFINITY) return;
        const unsigned long long entry = pick_entry(x, t);
        if (entry < last) mine = max_u64(mine, entry);
      };
      again(0u, [&](int t, float y) { look(t, y); });
      for (int t = tid; t < r.V; t += kThreads) look(t, free_value(t));
      mine = warp_max_u64(mine);
      if (lane == 0) s.red[warp] = mine;
      __syncthreads();
      unsigned long long all = 0ull;
      for (int w = 0; w < kWarps; ++w) all = max_u64(all, s.red[w]);
      if (tid == 0) s.best[k] = all;
      last = all;  // (0, when nothing is left: then nothing is below it)
      __syncthreads();
    }
  }
  store_rest();
  if (warp > 0) return;
  const unsigned long long mine = lane < r.K ? s.best[lane] : 0ull;
  int token = mine != 0ull ? static_cast<int>(~static_cast<uint32_t>(mine)) : -1;
  const float value = mine != 0ull ? pick_value(static_cast<uint32_t>(mine >> 32)) : -INFINITY;
  // fewer than K tokens above -inf: all of them are here, and the lowest others follow
  int found = __popc(__ballot_sync(0xffffffffu, mine != 0ull));
  for (int t = 0; found < r.K; ++t)
    if (__ballot_sync(0xffffffffu, token == t) == 0u) {
      if (lane == found) token = t;
      ++found;
    }
  if (lane < r.K) {
    r.cand[static_cast<int64_t>(m) * r.K + lane] = token;
    r.unary[static_cast<int64_t>(m) * r.K + lane] = value;
  }
}

// Sizes, and where each part lies in the workspace.
struct PickPlan {
  int windows, cap, words, tiles;
  size_t bits, named, names, request, line, keys, total;
};
PickPlan pick_plan(int M, int V, int B, bool ragged, int max_len, bool tokens, int n_bias, int K) {
  PickPlan p{};
  const int most = max_len + (tokens ? kTreeRows : 0) + n_bias;
  p.windows = most > 0 ? (V + kWindow - 1) / kWindow : 0;
  p.cap = std::min(kWindow, most);
  p.words = (V + 31) / 32;
  p.tiles = (V + 7 + kTile - 1) / kTile;  // (wherever in sixteen bytes a row begins)
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t parts = static_cast<size_t>(B) * p.windows;
  p.bits = take(p.windows > 0 ? static_cast<size_t>(B) * p.words * 4 : 0);
  p.named = take(parts * 4);
  p.names = take(parts * p.cap * sizeof(uint2));
  p.request = take(ragged ? static_cast<size_t>(M) * 4 : 0);
  p.line = take(tokens ? static_cast<size_t>(M) * 8 : 0);
  p.keys = take(K > 0 ? static_cast<size_t>(M) * p.tiles * 128 : 0);
  p.total = at;
  return p;
}

// bits, a base for four words of them, counters
constexpr int kStreamShared = 112 * 1024;  // (two CTAs an SM)
constexpr int kSelectShared = (1 << 22) / kTile * 4 + 8 + 8192 * 4;  // marks, and kept values

template <typename T, int kThreads>
int launch_select(PickArgs a, cudaStream_t st) {
  static unsigned done = 0;
  if (!ensure_smem_attr(logits_select_kernel<T, kThreads>, kSelectShared, &done))
    return fail(DFLASH2_ERR_CUDA, "cudaFuncSetAttribute failed (logits)");
  // named tokens' values, kept for the second look (those histories: 47 us, with none kept 52)
  a.kept = std::min(a.windows * a.cap, 8 * kThreads);
  const cudaError_t e = launch_pdl(logits_select_kernel<T, kThreads>, dim3(static_cast<unsigned>(a.r.M)), dim3(kThreads),
                                   static_cast<size_t>(a.tiles + a.kept) * 4, st, nullptr, 0, a);
  return e == cudaSuccess ? DFLASH2_OK : fail(DFLASH2_ERR_CUDA, "logits launch failed: %s", cudaGetErrorString(e));
}

template <typename T>
int launch_pick_t(PickArgs& a, cudaStream_t st) {
  static unsigned done = 0;
  if (!ensure_smem_attr(logits_stream_kernel<T>, kStreamShared, &done))
    return fail(DFLASH2_ERR_CUDA, "cudaFuncSetAttribute failed (logits)");
  const int quads = (std::min(a.r.V, kWindow) + 127) / 128;
  // (a multiple of 32, and one word more of each kind)
  const int counters = (a.cap + 63) / 32 * 32, shared = quads * 20 + counters / 2 * 4 + counters / 32 * 4;
  // (counters in shared memory, of 16 bits: 63 rows with histories of 30000 tokens take 47 us, with counters in the
  // workspace 57; where counts or places do not fit they are there)
  a.counters = a.windows > 0 && a.r.max_len <= 0xffff && shared <= kStreamShared ? counters : 0;
  const cudaError_t e = launch_pdl(logits_stream_kernel<T>, dim3(static_cast<unsigned>(a.stream_ctas + a.other_ctas)),
                                   dim3(kStreamThreads), a.windows == 0 ? 0 : static_cast<size_t>(a.counters > 0 ? shared : quads * 20), st,
                                   nullptr, 0, a);
  if (e != cudaSuccess) return fail(DFLASH2_ERR_CUDA, "logits launch failed: %s", cudaGetErrorString(e));
  if (a.r.K == 0 && a.windows == 0) return DFLASH2_OK;
  // Threads a row. Up to a row an SM, the row's own time counts: 1024 (15 rows of 248320 tokens take 14.4 us, with 512
  // 15.8, with 256 18.6; 63 rows with histories of 30000 tokens 47, 66, 85). Up to three 512 (288 tree rows of 248320 tokens
  // 38.5 us; with 1024 41.1, with 256 40.7). Above them the number of rows in flight: 256 (960 rows 162 us; with 512 163,
  // with 1024 184; 4096 rows of 8000 tokens 97, with 512 126), and 128 where a row's keys are few (16384 rows of 1000 tokens
  // 64 us, with 256 104; 4096 of 8000 52 and 59; but 600 of 32771 18.9 and 18.2, 960 of 248320 194 and 162).
  const int sms = sm_count();
  if (a.r.M <= sms) return launch_select<T, 1024>(a, st);
  if (a.r.M <= 3 * sms) return launch_select<T, 512>(a, st);
  return a.tiles > 16 ? launch_select<T, 256>(a, st) : launch_select<T, 128>(a, st);
}

}  // namespace

size_t logits_topk_workspace(int M, int V, int B, bool ragged, int max_len, bool tokens, int n_bias, int K) {
  return pick_plan(M, V, B, ragged, max_len, tokens, n_bias, K).total;
}

int launch_logits_topk(const LogitsTopk& r, cudaStream_t st) {
  const PickPlan p = pick_plan(r.M, r.V, r.B, r.row_off != nullptr, r.max_len, r.tokens != nullptr, r.n_bias, r.K);
  PickArgs a{};
  a.r = r;
  a.each = r.row_off == nullptr ? r.M / r.B : 0;
  a.windows = p.windows; a.cap = p.cap; a.words = p.words; a.tiles = p.tiles;
  uint8_t* ws = static_cast<uint8_t*>(r.workspace);
  a.bits = reinterpret_cast<uint32_t*>(ws + p.bits);
  a.named = reinterpret_cast<int*>(ws + p.named);
  a.names = reinterpret_cast<uint2*>(ws + p.names);
  a.request = reinterpret_cast<int*>(ws + p.request);
  a.line = reinterpret_cast<uint64_t*>(ws + p.line);
  a.keys = reinterpret_cast<uint32_t*>(ws + p.keys);
  a.err = device_error_word();
  if (a.err == nullptr) return fail(DFLASH2_ERR_CUDA, "no device error word");
  // tiles a warp: one while the SMs have warps left for the next (two CTAs each). (15 rows of 248320 tokens: one and four
  // take 14.4 and 14.2 us; 960 rows 166.5 and 162, 288 rows under masks 48 and 38.)
  a.warp_tiles = static_cast<int>(std::min<int64_t>(kStreamTiles, 1 + static_cast<int64_t>(r.M) * a.tiles / (2 * kStreamWarps * sm_count())));
  a.row_warps = (a.tiles + a.warp_tiles - 1) / a.warp_tiles;
  a.stream_ctas = (r.M * a.row_warps + kStreamWarps - 1) / kStreamWarps;
  a.other_ctas = r.B * p.windows + (r.row_off != nullptr ? (r.M + kStreamThreads - 1) / kStreamThreads : 0);
  return r.dtype == DFLASH2_F32 ? launch_pick_t<float>(a, st) : launch_pick_t<__nv_bfloat16>(a, st);
}

}  // namespace dfl
