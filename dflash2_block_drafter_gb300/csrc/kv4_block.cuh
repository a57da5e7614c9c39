// What the kernels of attention over the 4-bit cache share: a call's arguments, the line of all tiles and its ranges,
// powers of two, and the conversion of codes and rows to fp16 operands.
#pragma once

#include <cuda_fp16.h>

#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace dfl {
namespace {

constexpr int kBTileLog = 7, kBTile = 1 << kBTileLog;  // keys per tile
constexpr int kBSoftWarps = 8, kBDeqWarps = 8, kBMmaWarp = 16, kBCopyWarp = 18;  // two each
constexpr int kBSoft = 32 * kBSoftWarps;    // softmax threads
constexpr int kBThreads = 640;
constexpr float kBLift = 7.f;               // a row's largest probability is 2^7 when its reference is set, and may
constexpr float kBSlack = 15.f;             // grow to 2^15 (fp16 holds 2^15, and steps of 2^-24)
constexpr float kBSumUnit = 0x1p-12f;       // of the sums: 2^31 keys of the smallest values' factor, 2^-93, stay finite
constexpr float kBUnseen = 3e38f;           // minus the reference of a row that has seen no key: any score passes it
constexpr uint32_t kBPow2Low = 9u << 23;     // 2^-118: powers of two of keys go no lower
constexpr uint32_t kBPow2LowQV = 27u << 23;  // 2^-100: nor those of queries and values
constexpr float kBLiftQ = 16384.f;           // a query row's largest value is in [2^14, 2^15)
constexpr float kBPadding = -1e30f;         // of a row that does not exist: no score passes it, and it counts nothing

struct BlockArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const uint8_t* cache;
  const int32_t *table, *ctx;
  const __nv_bfloat16 *k_new, *v_new;
  int64_t new_stride;
  const int32_t* parents;  // [B][G], of trees
  int B, G, Hq, Hkv, R, r_magic, rows, tile_rows, row_tiles, page_shift, num_pages, width, cap, causal, window;
  float scale_log2;
  __nv_bfloat16* out;
  float* part_o;    // [CTA][2][N][D]
  float2* part_ml;  // [CTA][2][N]
  unsigned long long* flags;  // [CTA]
  unsigned long long call, ctas_inverse;  // (the latter floor((2^64 - 1) / CTAs))
  int* err;
};

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// One MMA whose descriptors share the upper words; `first` overwrites the accumulator.
template <bool first>
__device__ __forceinline__ void mma_lean(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t a_hi, uint32_t b_hi,
                                         uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(a_hi), "r"(b_hi), "r"(idesc), "n"(first ? 0 : 1)
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// (Suspended, not spinning: the issue slots belong to the warps that work.)
__device__ __forceinline__ void wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_suspend(bar, parity, 20000))
    if (*abort_flag != 0 || globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      atomicCAS(err, 0, static_cast<int>(DFLASH2_ERR_TIMEOUT));
      break;
    }
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Token of query row r (r / R): r < 64 R, so ceil(2^20 / R) r is below 2^27 and exact after the shift.
__device__ __forceinline__ int row_token(const BlockArgs& a, int r) { return (r * a.r_magic) >> 20; }

// The keys of one sequence: [lo, hi) cached ones that some row sees, in `cached` tiles from lo / 128 on,
// then (own) one tile of its own rows. At least one tile, so that every item is visited.
struct BlockSeq {
  int L, base, lo, hi, cached, tiles;
};
__device__ __forceinline__ BlockSeq block_seq(const BlockArgs& a, int b) {
  BlockSeq s;
  const int own = a.k_new != nullptr ? 1 : 0;
  s.L = min(max(__ldg(a.ctx + b), 0), a.cap);  // (block_range records a length outside)
  s.base = s.L + (own - 1) * a.G;
  s.lo = a.window > 0 ? max(0, min(s.L, s.base - a.window + 1)) : 0;
  s.hi = a.causal ? max(0, min(s.L, s.base + a.G)) : s.L;
  s.cached = s.hi > s.lo ? ((s.hi - 1) >> kBTileLog) - (s.lo >> kBTileLog) + 1 : 0;
  s.tiles = max(1, s.cached + own);
  return s;
}

// floor(x / d) for a quotient below 2^22: the float estimate is off by one at most. (A 64-bit division is some
// hundred instructions.)
__device__ __forceinline__ int small_quotient(long long x, long long d) {
  int q = static_cast<int>(static_cast<float>(x) / static_cast<float>(d));
  if (q * d > x) --q;
  if ((q + 1) * d <= x) ++q;
  return q;
}

// The line of all units (a tile, or a part of an item's setup), cut into n ranges that differ by one unit at
// most and of which none is empty: range c starts at floor(c total / n).
struct BlockLine {
  long long total, q;  // q, rem: total over n
  int rem, n;
  __device__ __forceinline__ void set(long long total_, int ctas, unsigned long long ctas_inverse) {
    total = total_;
    n = total < ctas ? static_cast<int>(total) : ctas;
    q = n < ctas ? 1 : static_cast<long long>(__umul64hi(total, ctas_inverse));  // (one too small at most)
    if (total - q * n >= n) ++q;
    rem = static_cast<int>(total - q * n);
  }
  __device__ __forceinline__ long long start(int c) const { return q * c + rem * c / n; }
  // the range that holds unit g: the one c with start(c) <= g < start(c + 1)
  __device__ __forceinline__ int range_of(long long g) const {
    int c = small_quotient(g, q);  // at least the range: no range is shorter than q
    c = min(c, n - 1);
    if (rem > 0) {
      c = min(c, static_cast<int>(static_cast<float>(g) * static_cast<float>(n) / static_cast<float>(total)) + 1);
      while (start(c) > g) --c;
    }
    return c;
  }
};

// A CTA's range of the line.
struct BlockRange {
  BlockLine line;
  long long first, count;         // in units
  int b;                          // the sequence of its first unit, and that unit's place among the sequence's
  long long in_seq;
};
// A warp's work (all lanes call it): sums the sequences' units and finds range `c` of `ctas`. A lane sums a run of
// sequences; the run that holds the range's start is then walked 32 sequences at a time.
__device__ __forceinline__ BlockRange block_range(const BlockArgs& a, int setup, int c, int ctas) {
  const int lane = threadIdx.x & 31, hr = a.Hkv * a.row_tiles;
  const int per = (a.B + 31) / 32;
  auto prefix = [&](long long x) {  // over the lanes, this one's included
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, x, m);
      if (lane >= m) x += v;
    }
    return x;
  };
  long long mine = 0;
  for (int b = lane * per; b < min(a.B, (lane + 1) * per); ++b) {
    const int len = __ldg(a.ctx + b);
    if (len < 0 || len > a.cap) atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_INVALID_ARG));
    mine += block_seq(a, b).tiles + setup;
  }
  mine *= hr;
  long long inc = prefix(mine);
  BlockRange r;
  r.line.set(__shfl_sync(0xffffffffu, inc, 31), ctas, a.ctas_inverse);
  r.first = r.line.start(c);
  r.count = c < r.line.n ? r.line.start(c + 1) - r.first : 0;
  r.b = -1;
  r.in_seq = 0;
  uint32_t hit = __ballot_sync(0xffffffffu, r.first >= inc - mine && r.first < inc);
  if (hit == 0u) return r;  // (more CTAs than units)
  const int run = __ffs(hit) - 1;
  long long before = __shfl_sync(0xffffffffu, inc - mine, run);
  if (per == 1) {
    r.b = run;
    r.in_seq = r.first - before;
    return r;
  }
  for (int b0 = run * per; b0 < min(a.B, (run + 1) * per); b0 += 32) {
    const int b = b0 + lane;
    mine = b < min(a.B, (run + 1) * per) ? static_cast<long long>(block_seq(a, b).tiles + setup) * hr : 0;
    inc = before + prefix(mine);
    hit = __ballot_sync(0xffffffffu, r.first >= inc - mine && r.first < inc);
    if (hit != 0u) {
      const int at = __ffs(hit) - 1;
      r.b = b0 + at;
      r.in_seq = r.first - __shfl_sync(0xffffffffu, inc - mine, at);
      return r;
    }
    before = __shfl_sync(0xffffffffu, inc, 31);
  }
  return r;
}

// Walks a range piece by piece: piece = consecutive tiles [j0, j1) of one item (sequence b, head, row tile rt),
// none empty.
template <int kSetup>
struct BlockWalk {
  int left;  // units (a cache that fits the memory has far fewer tiles than 2^31)
  int b, head, rt, j0, j1;
  long long start;  // the item's first unit
  BlockSeq seq;
  __device__ __forceinline__ BlockWalk(const BlockArgs& a, const BlockRange& r) {
    left = static_cast<int>(r.count);
    b = r.b;
    j1 = -1;
    if (left <= 0) return;
    seq = block_seq(a, b);
    const int hr = small_quotient(r.in_seq, seq.tiles + kSetup);
    head = hr / a.row_tiles;
    rt = hr - head * a.row_tiles;
    const int u = static_cast<int>(r.in_seq - static_cast<long long>(hr) * (seq.tiles + kSetup));
    start = r.first - u;
    enter(u);
  }
  // at unit u of the item; a range that ends within the setup has nothing left
  __device__ __forceinline__ void enter(int u) {
    j0 = max(0, u - kSetup);
    j1 = min(seq.tiles, u + left - kSetup);
    left -= min(left, seq.tiles + kSetup - u);
    if (j1 <= j0) j1 = -1;
  }
  __device__ __forceinline__ bool valid() const { return j1 > 0; }
  __device__ __forceinline__ void next(const BlockArgs& a) {
    if (left <= 0) {
      j1 = -1;
      return;
    }
    start += seq.tiles + kSetup;
    if (++rt == a.row_tiles) {
      rt = 0;
      if (++head == a.Hkv) {
        head = 0;
        seq = block_seq(a, ++b);
      }
    }
    enter(0);
  }
};

// The ranges [c0, c1] that hold the tiles of the item that starts at unit `start`.
struct BlockParts {
  int c0, c1;
  int group;  // parts that are joined first: the smallest number whose square is at least all
  __device__ __forceinline__ BlockParts(const BlockLine& line, long long start, int setup, int tiles)
      : c0(line.range_of(start + setup)), c1(line.range_of(start + setup + tiles - 1)), group(1) {
    const int all = c1 - c0 + 1;
    if (all <= 8) group = all;
    while (group * group < all) ++group;
  }
  // range c ends a group of parts, and not the item
  __device__ __forceinline__ bool leads(int c) const { return c < c1 && group > 1 && (c - c0) % group == group - 1; }
  // what range c joins, c itself the last: if it leads, its group; if it ends the item, the groups before
  // its own and then its own group's parts
  __device__ __forceinline__ int inputs(int c) const { return c < c1 ? group : (c - c0) / group + (c - c0) % group + 1; }
  __device__ __forceinline__ int input(int c, int p) const {
    if (c < c1) return c - (group - 1) + p;
    const int groups = (c - c0) / group;
    return p < groups ? c0 + (p + 1) * group - 1 : c0 + groups * group + (p - groups);
  }
  // where the part of range c lies: the first part is a range's last piece, the others a range's first
  __device__ __forceinline__ int slot(int c) const { return c * 2 + (c == c0 ? 1 : 0); }
};

// 2^floor(log2 x) of a positive float (bits below the exponent dropped), kept inside [low, 2^118].
__device__ __forceinline__ float pow2_of(float x, uint32_t low = kBPow2Low) {
  const uint32_t u = __float_as_uint(x) & 0x7f800000u;
  return __uint_as_float(min(max(u, low), 0x7a800000u));
}
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float(0x7f000000u - __float_as_uint(p)); }

// Channels (0, 4), (1, 5), (2, 6), (3, 7) of a word of codes: scale * code + bias. A code masked out at
// bit 0 or 4 of a half-word is the fp16 subnormal n 2^-24 or n 2^-20; s24, s20: scale 2^24, scale 2^20.
__device__ __forceinline__ uint4 dequant_word(uint32_t w, __half2 s24, __half2 s20, __half2 b) {
  const uint32_t h = w >> 8;
  const uint32_t n[4] = {w & 0x000F000Fu, w & 0x00F000F0u, h & 0x000F000Fu, h & 0x00F000F0u};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __hfma2((i & 1) ? s20 : s24, *reinterpret_cast<const __half2*>(&n[i]), b);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// Eight bf16 channels times a factor, in the same order.
__device__ __forceinline__ uint4 convert_word(const uint4& u, float f) {
  float x[8];
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __bfloat1622float2(as_bf162(w[i]));
    x[2 * i] = v.x * f;
    x[2 * i + 1] = v.y * f;
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __floats2half2_rn(x[i], x[i + 4]);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// The largest magnitude as the bits of an fp32 number (they compare as integers, NaN above infinity).
__device__ __forceinline__ uint32_t max_abs8(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  return m << 16;
}
constexpr uint32_t kBInfinity = 0x7f800000u;
// one of a pair of bf16 is infinite or NaN
__device__ __forceinline__ bool pair_not_finite(uint32_t p) {
  return (p & 0x7f80u) == 0x7f80u || (p & 0x7f800000u) == 0x7f800000u;
}

// A row's (scale, bias) pairs as operands of dequant_word: half2 (scale 2^24, bias) over the row's power
// of two, and that power times 2^7 (the factor to undo it).
template <int kGroups>
__device__ __forceinline__ float row_params(const uint32_t (&par)[2], uint32_t (&out)[2], uint32_t low) {
  float2 p[2];
  float m = 0.f;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    p[g] = __bfloat1622float2(as_bf162(par[g]));
    m = fmaxf(m, fmaxf(fabsf(p[g].y), fabsf(fmaf(15.f, p[g].x, p[g].y))));
  }
  const float f = pow2_of(m, low), inv = pow2_inverse(f) * 0.0078125f;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const __half2 h = __floats2half2_rn(p[g].x * inv * 16777216.f, p[g].y * inv);
    out[g] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return f * 128.f;
}

// Where the eight channels of code word w of a row (w = D / 32 chunks of four words) lie among the operands'
// 16-byte pieces, the same for K, Q and V: with D = 128 the four chunks' words k of a key, and those of its
// neighbour, fall on eight different pieces of the swizzled 128 bytes, so neither the loads of codes
// (two rows of 64 contiguous bytes a phase) nor the stores conflict.
template <int D>
__device__ __forceinline__ constexpr int piece_of_word(int w) {
  return D == 128 ? ((w >> 1) & 1) * 8 + (w >> 2) * 2 + (w & 1) : w;
}
template <int D>
__device__ __forceinline__ constexpr int word_of_piece(int p) {
  return D == 128 ? ((p & 7) >> 1) * 4 + (p >> 3) * 2 + (p & 1) : p;
}

// Operand descriptor of MN-major fp16 tiles: 64-wide chunks 16 KB apart, 8 keys = 1024 bytes.
__device__ __forceinline__ uint64_t desc_keys_sw128(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(kBTile * 128 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

// A call's arguments but for the workspace's. False: no device error word.
inline bool block_args(const Kv4Attention& r, int ctas, int row_tiles, int tile_rows, BlockArgs& a) {
  a.q = static_cast<const __nv_bfloat16*>(r.q);
  a.q_stride = r.q_stride;
  a.cache = static_cast<const uint8_t*>(r.cache);
  a.table = r.table;
  a.ctx = r.ctx;
  a.k_new = static_cast<const __nv_bfloat16*>(r.k_new);
  a.v_new = static_cast<const __nv_bfloat16*>(r.v_new);
  a.new_stride = r.new_stride;
  a.parents = r.parents;
  a.B = r.B; a.G = r.G; a.Hq = r.Hq; a.Hkv = r.Hkv;
  a.R = r.Hq / r.Hkv;
  a.r_magic = ((1 << 20) + a.R - 1) / a.R;
  a.rows = r.G * a.R;
  a.tile_rows = tile_rows;
  a.row_tiles = row_tiles;
  while ((1 << a.page_shift) < r.page_size) ++a.page_shift;
  a.num_pages = r.num_pages;
  a.width = r.max_pages;
  a.cap = r.max_pages * r.page_size;  // (below 2^31: checked)
  a.causal = r.causal;
  a.window = r.window;
  a.scale_log2 = r.scale * 1.4426950408889634f;
  a.out = static_cast<__nv_bfloat16*>(r.out);
  a.ctas_inverse = ~0ull / static_cast<unsigned long long>(ctas);
  a.err = device_error_word();
  return a.err != nullptr;
}

}  // namespace
}  // namespace dfl
