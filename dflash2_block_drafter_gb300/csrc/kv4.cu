// The 4-bit key/value cache of the drafter's attention sublayer: writing rows, reading rows back, and
// attention over it (dflash2.ts #contextKV and #block: the block's queries attend to the context's
// keys and values and, bidirectionally, to the block's own; MAX DFlash2Qwen3_5.materialize).
//
// Quantisation, per token, head and group of 64 channels (affine, as dflash2.ts quantizedWeight's):
//   bias = bf16(min x), scale = bf16((max x - min x) / 15), code = clamp(round((x - bias) / scale), 0, 15)
// in IEEE fp32 with ties to even (scale = 0: code 0).
//
// Attention of one sequence: key i < L is cached row i, key L + j its own row j (unquantised, N of
// them, or none); query row t stands at position p_t = L + N - G + t and sees key i if i < L + N, and
// i <= p_t (causal), and i > p_t - window (window > 0);
//   out_t = sum_i softmax_i(scale q_t . k_i) v_i over the keys it sees, 0 if it sees none.
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

// ---------------------------------------------------------------- attention on warp-level MMAs
// One CTA of four warps takes 16 query rows of one (sequence, key/value head) (rows t R + j: token t,
// query head j of the R that share the head) and one of `ns` ranges of its keys. Each warp walks its
// own units of 32 keys (two granules) with a private ring of bulk copies, so that warps never wait
// for one another:
//   S = Q K^T by m16n8k16: the key fragment of a lane is one contiguous run of a cached row (channels
//       D/4 (lane % 4) ..), so the reduction index is permuted and Q is permuted alike;
//   running maximum m and sum l per row (fp32), P = exp2(S - m) rounded to bf16 (the MMA's operand;
//       l sums the unrounded values);
//   O += P V: a value fragment pairs two tokens of one channel. Two byte permutes put the halves of
//       two tokens' words side by side, and then a shift and a mask give such pairs directly.
// The four warps' (m, l, O) join in shared memory; with ns > 1 the ranges' partial results go through
// the workspace to kv4_join_kernel.
constexpr int kAWarps = 4;
constexpr int kAUnit = 32;    // keys per unit
constexpr int kAStages = 3;   // units in flight per warp
constexpr uint64_t kADrainNs = 100000000ull;

struct KvAttnArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const uint8_t* cache;
  const int32_t *table, *ctx;
  const __nv_bfloat16 *k_new, *v_new;
  int64_t new_stride;
  int B, G, Hq, Hkv, R, rows, row_tiles, page_shift, num_pages, width, causal, window, ns;
  float scale_log2;  // softmax scale x log2(e)
  __nv_bfloat16* out;
  float* part_o;   // [B][Hkv][rows][ns][D], relative to the range's maximum
  float2* part_ml; // [B][Hkv][rows][ns] (maximum in the log2 domain, sum)
  int* err;
};

__device__ __forceinline__ void mma_16x8x16_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Cached tokens of sequence b (a length outside [0, width * page_size] is recorded and clamped).
__device__ __forceinline__ int kv_context(const KvAttnArgs& a, int b) {
  const int n = a.ctx[b];
  const int64_t cap = static_cast<int64_t>(a.width) << a.page_shift;
  if (n < 0 || n > cap) {
    atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_INVALID_ARG));
    return n < 0 ? 0 : static_cast<int>(cap);
  }
  return n;
}

// What the keys of a 16-row tile need: positions of its rows and the bounds of what they see.
struct KvSpan {
  int L, keys;      // cached keys, all keys
  int base;         // position of query token 0
  int lo, hi;       // cached keys that some row of the tile sees: [lo, hi)
};
__device__ __forceinline__ KvSpan kv_span(const KvAttnArgs& a, int b, int t_first, int t_last) {
  KvSpan s;
  s.L = kv_context(a, b);
  s.keys = s.L + (a.k_new != nullptr ? a.G : 0);
  s.base = s.keys - a.G;
  // (positions fit in int: the context is below 2^31 - 64 tokens, checked on the host)
  s.lo = a.window > 0 ? max(0, min(s.L, s.base + t_first - a.window + 1)) : 0;
  s.hi = a.causal ? max(0, min(s.L, s.base + t_last + 1)) : s.L;
  return s;
}

// Scores of 32 keys -> P (bf16 A fragments), with the running maximum and sum and the rescaled O.
// `lo` / `hi`: the keys [lo, hi) relative to the unit's first that each of the lane's two rows sees.
template <int NT>
__device__ __forceinline__ void softmax_step(float (&s)[4][4], const int (&lo)[2], const int (&hi)[2], bool whole,
                                             float scale_log2, int c, float (&m)[2], float (&l)[2], float (&o)[NT][4],
                                             uint32_t (&p)[2][4]) {
  float mx[2] = {m[0], m[1]};
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = e >> 1;
      float v = s[j][e] * scale_log2;
      if (!whole) {
        const int key = j * 8 + 2 * c + (e & 1);
        if (key < lo[r] || key >= hi[r]) v = -INFINITY;
      }
      s[j][e] = v;
      mx[r] = fmaxf(mx[r], v);
    }
  bool grew = false;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
    mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
    grew |= mx[r] > m[r];
  }
  if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - mx[r]);
      m[r] = mx[r];
      l[r] *= f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][2 * r] *= f;
        o[n][2 * r + 1] *= f;
      }
    }
  }
  const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};  // a row that saw nothing yet
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[j][e] = ex2(s[j][e] - ref[e >> 1]);
      l[e >> 1] += s[j][e];
    }
    p[j >> 1][(j & 1) * 2] = pack_bf16(s[j][0], s[j][1]);
    p[j >> 1][(j & 1) * 2 + 1] = pack_bf16(s[j][2], s[j][3]);
  }
}

template <int D>
struct KvAttnCfg {
  static constexpr int kUnitBytes = 2 * 2 * KvLayout<D>::kGranuleBytes;  // [side][granule]
  static constexpr int kRing = kAStages * kUnitBytes;
  static constexpr int kOPitch = D + 4;
  static constexpr int kJoin = kAWarps * 16 * kOPitch * 4;
  static constexpr int kBody = kAWarps * kRing > kJoin ? kAWarps * kRing : kJoin;
  static constexpr int kSmem = kBody + kAWarps * 16 * 8 + kAWarps * kAStages * (8 + 4) + 64;
};

template <int D>
__global__ void __launch_bounds__(32 * kAWarps, 3) kv4_attn_kernel(const KvAttnArgs a) {
  using L = KvLayout<D>;
  using C = KvAttnCfg<D>;
  constexpr int NT = D / 8;     // channel tiles of O
  constexpr int WK = D / 32;    // words of a key row per lane
  constexpr int WV = D / 64;    // words of a value row per lane
  extern __shared__ __align__(128) uint8_t smem[];
  float2* ml = reinterpret_cast<float2*>(smem + C::kBody);                         // [warp][16]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ml + kAWarps * 16);                 // [warp][stage]
  uint32_t* there = reinterpret_cast<uint32_t*>(bars + kAWarps * kAStages);        // [warp][stage] granules that came

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int split = static_cast<int>(blockIdx.x) % a.ns;
  const int item = static_cast<int>(blockIdx.x) / a.ns;
  const int rt = item % a.row_tiles;
  const int head = (item / a.row_tiles) % a.Hkv;
  const int b = item / a.row_tiles / a.Hkv;
  uint8_t* ring = smem + warp * C::kRing;
  uint64_t* bar = bars + warp * kAStages;
  if (lane == 0)
    for (int s = 0; s < kAStages; ++s) mbar_init(smem_u32(&bar[s]), 1);
  fence_mbar_init();
  __syncwarp();
  pdl_trigger();
  pdl_wait();

  const int r_first = rt * 16;
  const int r_last = min(a.rows, r_first + 16) - 1;
  const KvSpan sp = kv_span(a, b, r_first / a.R, r_last / a.R);
  // this range's units: [u0, u1), warp w takes u0 + w, u0 + w + 4, ...
  const int u_lo = sp.lo / kAUnit, u_hi = (sp.hi + kAUnit - 1) / kAUnit;
  const int units = sp.hi > sp.lo ? u_hi - u_lo : 0;
  const int u0 = u_lo + static_cast<int>(static_cast<int64_t>(units) * split / a.ns) + warp;
  const int u1 = u_lo + static_cast<int>(static_cast<int64_t>(units) * (split + 1) / a.ns);

  // the copy of unit u: lanes 0-3 bring (granule lane & 1, side lane >> 1) if some row sees a key of it
  const int granules = (1 << a.page_shift) / kKvGranule;
  auto page_of = [&](int u) {
    const int gi = 2 * u + (lane & 1);
    if (lane >= 4 || u >= u1 || gi * kKvGranule >= sp.hi || gi * kKvGranule + kKvGranule <= sp.lo) return -1;
    const int page = a.table[static_cast<int64_t>(b) * a.width + ((gi * kKvGranule) >> a.page_shift)];
    if (page < 0 || page >= a.num_pages) {
      atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_BAD_INDEX));
      return -1;
    }
    return page;
  };
  auto issue = [&](int u, int stage, int page) {
    const uint32_t came = __ballot_sync(0xffffffffu, page >= 0);
    if (lane == 0) {
      there[warp * kAStages + stage] = came & 3u;
      mbar_arrive_expect_tx(smem_u32(&bar[stage]), static_cast<uint32_t>(__popc(came)) * L::kGranuleBytes);
    }
    __syncwarp();
    if (page >= 0) {
      const int in = (2 * u + (lane & 1)) & (granules - 1);
      const uint8_t* src = a.cache + (((static_cast<int64_t>(page) * a.Hkv + head) * 2 + (lane >> 1)) * granules + in) *
                                         static_cast<int64_t>(L::kGranuleBytes);
      bulk_load(smem_u32(ring + stage * C::kUnitBytes + lane * L::kGranuleBytes), src, L::kGranuleBytes,
                smem_u32(&bar[stage]));
    }
  };
#pragma unroll
  for (int s = 0; s < kAStages; ++s)
    if (u0 + s * kAWarps < u1) issue(u0 + s * kAWarps, s, page_of(u0 + s * kAWarps));
  int page_next = page_of(u0 + kAStages * kAWarps);

  // Q fragments: k step 2 w + h of word w pairs channels (8 w + 2 h, + 4) and (8 w + 2 h + 1, + 4) of the lane's run
  uint32_t q[2 * WK][4];
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int r = r_first + g + 8 * rr;
    const bool in = r < a.rows;
    const int t = in ? r / a.R : 0;
    const __nv_bfloat16* src =
        a.q + (static_cast<int64_t>(b) * a.G + t) * a.q_stride + (head * a.R + (in ? r - t * a.R : 0)) * D + c * (D / 4);
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(src + 8 * w)) : make_uint4(0u, 0u, 0u, 0u);
      q[2 * w][rr] = __byte_perm(u.x, u.z, 0x5410);
      q[2 * w][2 + rr] = __byte_perm(u.x, u.z, 0x7632);
      q[2 * w + 1][rr] = __byte_perm(u.y, u.w, 0x5410);
      q[2 * w + 1][2 + rr] = __byte_perm(u.y, u.w, 0x7632);
    }
  }
  // the keys [row_lo, row_hi) that the lane's two rows see
  int row_lo[2], row_hi[2];
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const int r = min(r_first + g + 8 * rr, a.rows - 1);
    const int pos = sp.base + r / a.R;
    row_lo[rr] = a.window > 0 ? pos - a.window + 1 : 0;
    row_hi[rr] = a.causal ? min(sp.keys, pos + 1) : sp.keys;
  }
  const int all_lo = a.window > 0 ? sp.base + r_last / a.R - a.window + 1 : 0;   // seen by every row of the tile
  const int all_hi = min(sp.L, a.causal ? sp.base + r_first / a.R + 1 : sp.L);

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

  int stage = 0;
  uint32_t phase = 0;
  int done = 0;
  for (int u = u0; u < u1; u += kAWarps, ++done) {
    if (!mbar_wait_bounded(smem_u32(&bar[stage]), phase, nullptr, kWaitLimitNs)) {
      if (lane == 0) atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_TIMEOUT));
      for (int s = 0; s < kAStages; ++s)  // copies in flight land before the CTA leaves
        if (s != stage && u + kAWarps * ((s - stage + kAStages) % kAStages) < u1)
          mbar_wait_bounded(smem_u32(&bar[s]), s > stage ? phase : phase ^ 1u, nullptr, kADrainNs);
      break;
    }
    const uint8_t* kt = ring + stage * C::kUnitBytes;
    const uint8_t* vt = kt + 2 * L::kGranuleBytes;
    const int key0 = u * kAUnit;
    const uint32_t came = there[warp * kAStages + stage];
    const bool whole = came == 3u && key0 >= all_lo && key0 + kAUnit <= all_hi;
    float s[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* gr = kt + (j >> 1) * L::kGranuleBytes;
      const int token = (j & 1) * 8 + g;
      uint32_t w[WK];
      if (WK == 4) {
        const uint4 u4 = *reinterpret_cast<const uint4*>(gr + token * L::kRow + c * 16);
        w[0] = u4.x; w[1] = u4.y; w[WK - 2] = u4.z; w[WK - 1] = u4.w;
      } else {
        const uint2 u2 = *reinterpret_cast<const uint2*>(gr + token * L::kRow + c * 8);
        w[0] = u2.x; w[1] = u2.y;
      }
      const __nv_bfloat162 sb = *reinterpret_cast<const __nv_bfloat162*>(
          gr + L::kCodes + (token * L::kGroups + (L::kGroups == 2 ? c >> 1 : 0)) * 4);
      const __nv_bfloat162 s2 = __low2bfloat162(sb), b2 = __high2bfloat162(sb);
      s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int i = 0; i < WK; ++i) {
        mma_16x8x16_bf16(s[j], q[2 * i], kv_value(w[i], s2, b2), kv_value(w[i] >> 4, s2, b2));
        mma_16x8x16_bf16(s[j], q[2 * i + 1], kv_value(w[i] >> 8, s2, b2), kv_value(w[i] >> 12, s2, b2));
      }
    }
    int lo[2], hi[2];
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      lo[rr] = row_lo[rr] - key0;
      hi[rr] = min(row_hi[rr], sp.L) - key0;
      if (!(came & 1u)) lo[rr] = max(lo[rr], 16);
      if (!(came & 2u)) hi[rr] = min(hi[rr], 16);
    }
    uint32_t p[2][4];
    softmax_step(s, lo, hi, whole, a.scale_log2, c, m, l, o, p);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const uint8_t* gr = vt + kk * L::kGranuleBytes;
      uint32_t w[4][WV], par[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // tokens 2c, 2c + 1, 2c + 8, 2c + 9
        const int token = 2 * c + (i & 1) + (i >> 1) * 8;
        if (WV == 2) {
          const uint2 u2 = *reinterpret_cast<const uint2*>(gr + token * L::kRow + g * 8);
          w[i][0] = u2.x;
          w[i][WV - 1] = u2.y;
        } else {
          w[i][0] = *reinterpret_cast<const uint32_t*>(gr + token * L::kRow + g * 4);
        }
        par[i] = *reinterpret_cast<const uint32_t*>(
            gr + L::kCodes + (token * L::kGroups + (L::kGroups == 2 ? g >> 2 : 0)) * 4);
        // rows that no query sees may hold anything: they count as zeros
        if (!whole) {
          const int key = key0 + kk * 16 + token;
          if (!((came >> kk) & 1u) || key < sp.lo || key >= sp.hi) par[i] = 0u;
        }
      }
      const __nv_bfloat162 s0 = as_bf162(__byte_perm(par[0], par[1], 0x5410));
      const __nv_bfloat162 b0 = as_bf162(__byte_perm(par[0], par[1], 0x7632));
      const __nv_bfloat162 s1 = as_bf162(__byte_perm(par[2], par[3], 0x5410));
      const __nv_bfloat162 b1 = as_bf162(__byte_perm(par[2], par[3], 0x7632));
#pragma unroll
      for (int wv = 0; wv < WV; ++wv) {
        const uint32_t x0 = __byte_perm(w[0][wv], w[1][wv], 0x5410), y0 = __byte_perm(w[0][wv], w[1][wv], 0x7632);
        const uint32_t x1 = __byte_perm(w[2][wv], w[3][wv], 0x5410), y1 = __byte_perm(w[2][wv], w[3][wv], 0x7632);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mma_16x8x16_bf16(o[wv * 8 + i], p[kk], kv_value(x0 >> (4 * i), s0, b0), kv_value(x1 >> (4 * i), s1, b1));
          mma_16x8x16_bf16(o[wv * 8 + 4 + i], p[kk], kv_value(y0 >> (4 * i), s0, b0), kv_value(y1 >> (4 * i), s1, b1));
        }
      }
    }
    __syncwarp();
    if (u + kAStages * kAWarps < u1) issue(u + kAStages * kAWarps, stage, page_next);
    page_next = page_of(u + (kAStages + 1) * kAWarps);
    if (++stage == kAStages) {
      stage = 0;
      phase ^= 1u;
    }
  }

  // the sequence's own rows, unquantised, by the last range's warps (32 keys each)
  if (a.k_new != nullptr && split == a.ns - 1) {
    for (int j0 = warp * kAUnit; j0 < a.G; j0 += kAWarps * kAUnit) {
      const __nv_bfloat16* kn = a.k_new + static_cast<int64_t>(b) * a.G * a.new_stride + head * D;
      const __nv_bfloat16* vn = a.v_new + static_cast<int64_t>(b) * a.G * a.new_stride + head * D;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      float s[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + j * 8 + g;
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
        for (int w = 0; w < WK; ++w) {
          const uint4 u = key < a.G ? __ldg(reinterpret_cast<const uint4*>(kn + key * a.new_stride + c * (D / 4) + 8 * w))
                                    : zero;
          mma_16x8x16_bf16(s[j], q[2 * w], __byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632));
          mma_16x8x16_bf16(s[j], q[2 * w + 1], __byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632));
        }
      }
      const int lo[2] = {row_lo[0] - sp.L - j0, row_lo[1] - sp.L - j0};
      const int hi[2] = {row_hi[0] - sp.L - j0, row_hi[1] - sp.L - j0};
      uint32_t p[2][4];
      softmax_step(s, lo, hi, false, a.scale_log2, c, m, l, o, p);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int wv = 0; wv < WV; ++wv) {
          uint32_t u[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = j0 + kk * 16 + 2 * c + (i & 1) + (i >> 1) * 8;
            const uint4 x = key < a.G
                                ? __ldg(reinterpret_cast<const uint4*>(vn + key * a.new_stride + g * (D / 8) + 8 * wv))
                                : zero;
            u[i][0] = x.x; u[i][1] = x.y; u[i][2] = x.z; u[i][3] = x.w;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t sel = (i & 1) ? 0x7632 : 0x5410;
            mma_16x8x16_bf16(o[wv * 8 + i], p[kk], __byte_perm(u[0][i >> 1], u[1][i >> 1], sel),
                             __byte_perm(u[2][i >> 1], u[3][i >> 1], sel));
          }
        }
    }
  }

  // ---- join the warps: O and (m, l) through shared memory (the rings are read out by now)
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  __syncthreads();
  float* ob = reinterpret_cast<float*>(smem) + warp * 16 * C::kOPitch;
#pragma unroll
  for (int rr = 0; rr < 2; ++rr)
#pragma unroll
    for (int cc = 0; cc < 2; ++cc)  // columns 2c and 2c + 1 of every channel tile: D / 8 channels in a row
#pragma unroll
      for (int n = 0; n < NT; n += 4)
        *reinterpret_cast<float4*>(ob + (g + 8 * rr) * C::kOPitch + (2 * c + cc) * (D / 8) + n) =
            make_float4(o[n][2 * rr + cc], o[n + 1][2 * rr + cc], o[n + 2][2 * rr + cc], o[n + 3][2 * rr + cc]);
  if (c == 0) {
    ml[warp * 16 + g] = make_float2(m[0], l[0]);
    ml[warp * 16 + g + 8] = make_float2(m[1], l[1]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * (D / 4); i += 32 * kAWarps) {
    const int row = i / (D / 4), col = (i % (D / 4)) * 4;
    const int r = r_first + row;
    if (r >= a.rows) continue;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAWarps; ++w) mm = fmaxf(mm, ml[w * 16 + row].x);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kAWarps; ++w) {
      const float2 x = ml[w * 16 + row];
      if (x.x == -INFINITY) continue;
      const float f = ex2(x.x - mm);
      const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                        (w * 16 + row) * C::kOPitch + col);
      sum += f * x.y;
      acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
    }
    if (a.ns > 1) {
      const int64_t at = ((static_cast<int64_t>(b) * a.Hkv + head) * a.rows + r) * a.ns + split;
      *reinterpret_cast<float4*>(a.part_o + at * D + col) = acc;
      if (col == 0) a.part_ml[at] = make_float2(mm, sum);
    } else {
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const int t = r / a.R;
      uint2 u;
      u.x = pack_bf16(acc.x * inv, acc.y * inv);
      u.y = pack_bf16(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(a.out + ((static_cast<int64_t>(b) * a.G + t) * a.Hq + head * a.R + r - t * a.R) * D + col) = u;
    }
  }
}

// Joins the ranges' partial results of every row: thread = 4 channels of one row.
template <int D>
__global__ void __launch_bounds__(256) kv4_join_kernel(const KvAttnArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = i / (D / 4);
  const int col = static_cast<int>(i % (D / 4)) * 4;
  if (row >= static_cast<int64_t>(a.B) * a.Hkv * a.rows) return;
  const int r = static_cast<int>(row % a.rows);
  const int64_t bh = row / a.rows;
  const int head = static_cast<int>(bh % a.Hkv);
  const int64_t b = bh / a.Hkv;
  float mm = -INFINITY;
  for (int s = 0; s < a.ns; ++s) mm = fmaxf(mm, a.part_ml[row * a.ns + s].x);
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < a.ns; ++s) {
    const float2 x = a.part_ml[row * a.ns + s];
    if (x.x == -INFINITY) continue;
    const float f = ex2(x.x - mm);
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + (row * a.ns + s) * D + col);
    sum += f * x.y;
    acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int t = r / a.R;
  uint2 u;
  u.x = pack_bf16(acc.x * inv, acc.y * inv);
  u.y = pack_bf16(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(a.out + ((b * a.G + t) * a.Hq + head * a.R + r - t * a.R) * D + col) = u;
}

// Ranges of keys per 16-row tile: enough CTAs to fill the SMs twice over (so that ragged contexts
// even out), none shorter than four units per warp at the longest context.
int attn_splits(int B, int Hkv, int row_tiles, int64_t max_ctx, int sms) {
  const int64_t items = static_cast<int64_t>(B) * Hkv * row_tiles;
  const int64_t want = (static_cast<int64_t>(sms) * 8 + items - 1) / items;
  const int64_t room = max_ctx / (kAWarps * kAUnit * 4);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, room, 64})));
}

template <int D>
int launch_attn_t(const KvAttnArgs& a, cudaStream_t st) {
  using C = KvAttnCfg<D>;
  static unsigned done = 0;
  auto kern = kv4_attn_kernel<D>;
  if (!ensure_smem_attr(kern, C::kSmem, &done)) return fail(DFLASH2_ERR_CUDA, "cudaFuncSetAttribute failed (attention)");
  const int64_t ctas = static_cast<int64_t>(a.B) * a.Hkv * a.row_tiles * a.ns;
  if (ctas > 0x7fffffffLL) return fail(DFLASH2_ERR_INVALID_ARG, "B=%d sequences are too many for one call", a.B);
  cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(32 * kAWarps), C::kSmem, st, nullptr, 0, a);
  if (e == cudaSuccess && a.ns > 1) {
    const int64_t n = static_cast<int64_t>(a.B) * a.Hkv * a.rows * (D / 4);
    e = launch_pdl(kv4_join_kernel<D>, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st, nullptr, 0, a);
  }
  return e == cudaSuccess ? DFLASH2_OK : fail(DFLASH2_ERR_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
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

size_t kv4_attention_workspace(int B, int G, int Hq, int Hkv, int D, int page_size, int max_pages, int sms) {
  const int rows = G * (Hq / Hkv);
  const int ns = attn_splits(B, Hkv, (rows + 15) / 16, static_cast<int64_t>(max_pages) * page_size, sms);
  if (ns == 1) return 0;
  const size_t parts = static_cast<size_t>(B) * Hkv * rows * ns;
  return parts * D * sizeof(float) + parts * sizeof(float2);
}

int launch_kv4_attention(const Kv4Attention& r, cudaStream_t st) {
  KvAttnArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(r.q);
  a.q_stride = r.q_stride;
  a.cache = static_cast<const uint8_t*>(r.cache);
  a.table = r.table;
  a.ctx = r.ctx;
  a.k_new = static_cast<const __nv_bfloat16*>(r.k_new);
  a.v_new = static_cast<const __nv_bfloat16*>(r.v_new);
  a.new_stride = r.new_stride;
  a.B = r.B;
  a.G = r.G;
  a.Hq = r.Hq;
  a.Hkv = r.Hkv;
  a.R = r.Hq / r.Hkv;
  a.rows = r.G * a.R;
  a.row_tiles = (a.rows + 15) / 16;
  a.page_shift = log2_of(r.page_size);
  a.num_pages = r.num_pages;
  a.width = r.max_pages;
  a.causal = r.causal;
  a.window = r.window;
  a.ns = attn_splits(r.B, r.Hkv, a.row_tiles, static_cast<int64_t>(r.max_pages) * r.page_size, sm_count());
  a.scale_log2 = r.scale * 1.4426950408889634f;
  a.out = static_cast<__nv_bfloat16*>(r.out);
  const size_t parts = static_cast<size_t>(r.B) * r.Hkv * a.rows * a.ns;
  a.part_o = static_cast<float*>(r.workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + parts * r.D);
  a.err = device_error_word();
  if (a.err == nullptr) return fail(DFLASH2_ERR_CUDA, "no device error word");
  return r.D == 64 ? launch_attn_t<64>(a, st) : launch_attn_t<128>(a, st);
}

}  // namespace dfl
