// Attention of trees with many rows over the 4-bit key/value cache: rows on the tensor core's 128-row side.
//
// kv4_attention.cu keeps keys on that side, so that few rows are not padded; from about a hundred rows a key/value head
// on, this kernel is the faster one. The same statement, precision and work line (kv4_block.cuh); what differs:
//
//   S [128 rows x 128 keys]  = Q [rows][D] . K tile [keys][D]^T       (both K-major, from shared memory)
//   O [128 rows x D]        += P [rows x keys] . V tile [keys][D]     (P from tensor memory, in place of S; V MN-major)
//
// A CTA works on two tiles of rows at once: while one's scores are made into probabilities, the tensor core runs the
// other's products, and a tile of codes is converted once for both. A softmax thread has one row, so maxima and sums need
// no other thread: the row's reference is raised, and its O rescaled, when a tile passes it by 2^8.
//
// Key and value rows go over powers of two as there, but one for each 32 keys of a tile where those rows lie within 2^4 of
// each other, so that a thread needs four pairs of factors a tile instead of 128. Tiles with rows further apart, with
// masks, or of the tree's own rows take a path that reads a factor a key.
//
// Ranges of the line leave partial results in the workspace. A range can end one item that earlier ones began; it says
// which there, and a second kernel joins the parts of these, a warp a row. (So no CTA waits for another.)
#include <algorithm>

#include "kv4_block.cuh"

namespace dfl {
namespace {

constexpr int kWRows = 128;        // of a tile of rows; two tiles
constexpr int kWSetup = 2;         // the change from one item to the next, in tiles
constexpr float kWSpread = 16.f;   // rows of 32 keys that share a factor differ by no more

template <int D>
struct WideCfg {
  using L = KvLayout<D>;
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kBTile * 128;    // fp16 [half][key or row][64]
  static constexpr int kOffV = 2 * kTileBytes, kOffQ = 4 * kTileBytes;
  static constexpr int kOffRaw = kOffQ + 2 * kTileBytes;       // [side][slot]: 64 keys of one side each
  static constexpr int kRaw = 4 * L::kGranuleBytes, kSlots = 3;
  static constexpr int kOffInfo = kOffRaw + 2 * kSlots * kRaw; // WideInfo [4]
  static constexpr int kOffLine = kOffInfo + 4 * 1120;         // uint64 [2][64]: of two items in turn
  static constexpr int kOffQs = kOffLine + 2 * kTreeRows * 8;  // float [2][128]: what a row's scores are multiplied by
  static constexpr int kOffBar = kOffQs + 2 * kWRows * 4;
  static constexpr int kSmem = 1024 + kOffBar + 384;
  // 640 x 96 registers at launch, shared out
  static constexpr int kSoftRegs = 144, kOtherRegs = 64;
};
struct WideInfo {
  float2 key[kBTile];     // each key's factor, its values' factor (-1: the key is not there, NaN: they are not finite)
  float k[4], v[4];       // those of each 32 keys,
  uint32_t there[4];      // which of them are there,
  uint32_t mixed_k[4], mixed_v[4];  // and whether they need factors of their own
};
static_assert(sizeof(WideInfo) <= 1120, "info");

// (Tensor-memory loads and stores are whole warps': each is preceded by a barrier of the warp, since nothing else keeps the
// compiler from leaving lanes apart after a condition of their own.)
__device__ __forceinline__ void tmem_ld32(uint32_t t, float (&x)[32]) {
  __syncwarp();
  tmem_ld_32x32b_x32(t, reinterpret_cast<uint32_t(&)[32]>(x));
}
__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t (&r)[16]) {
  __syncwarp();
  tmem_ld_32x32b_x16(t, r);
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&r)[16]) {
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t t, float (&x)[8]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  __syncwarp();
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}
__device__ __forceinline__ void tmem_st4(uint32_t t, const uint32_t (&r)[4]) {
  __syncwarp();
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// One MMA whose A operand lies in tensor memory.
template <bool first>
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(first ? 0 : 1)
      : "memory");
}

// One lane of a (converged) warp. (What it runs is known to be one thread's, so that the products' descriptors stay in
// uniform registers.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

// A row's largest value as a power of two (0: nothing but zeros), from its (scale, bias) pairs.
template <int kGroups>
__device__ __forceinline__ float row_largest(const uint32_t (&par)[2]) {
  float m = 0.f;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const float2 p = __bfloat1622float2(as_bf162(par[g]));
    m = fmaxf(m, fmaxf(fabsf(p.y), fabsf(fmaf(15.f, p.x, p.y))));
  }
  return m;
}

struct WideArgs {
  BlockArgs a;
  int2* entry;  // [CTA] the item that ends in its range and began in an earlier one (-1: none), and the range where
};

template <int D>
__global__ void __launch_bounds__(kBThreads, 1) kv4_wide_kernel(const WideArgs wa) {
  using C = WideCfg<D>;
  using L = KvLayout<D>;
  using Walk = BlockWalk<kWSetup>;
  const BlockArgs& a = wa.a;
  constexpr int NCH = D / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  auto info_of = [&](uint32_t it) { return reinterpret_cast<WideInfo*>(smem + C::kOffInfo + (it & 3u) * 1120); };
  uint64_t* tree_line = reinterpret_cast<uint64_t*>(smem + C::kOffLine);
  const uint32_t bars = smem_u32(smem + C::kOffBar);
  const uint32_t kfull = bars, kempty = bars + 16, vfull = bars + 32, vempty = bars + 48;  // [2] each: operand buffers
  const uint32_t sfull = bars + 64, pfull = bars + 96, odone = bars + 128;  // [row tile][buffer of scores]
  const uint32_t qfull = bars + 160;                                        // [row tile]
  const uint32_t raw_full = bars + 176, raw_empty = bars + 224;             // [side][3]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 272);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* came_s = tmem_slot + 2;  // [side][3]: the granules that came

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull + 8 * i, kBDeqWarps / 2);
      mbar_init(vfull + 8 * i, kBDeqWarps / 2);
      mbar_init(kempty + 8 * i, 1);
      mbar_init(vempty + 8 * i, 1);
      mbar_init(qfull + 8 * i, 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(sfull + 8 * i, 1);
      mbar_init(pfull + 8 * i, 4);
      mbar_init(odone + 8 * i, 1);
    }
    for (int i = 0; i < 6; ++i) {
      mbar_init(raw_full + 8 * i, 1);
      mbar_init(raw_empty + 8 * i, 2);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kBMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // S (then P) of a row tile: two buffers of 64 keys from column 0 or 128, O from 256 or 384
  pdl_trigger();
  pdl_wait();
  const BlockRange range = block_range(a, kWSetup, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
  // an item's rows: one tile of them, or two of equal size
  auto rows_of = [&](const Walk& w) { return min(a.tile_rows, a.rows - w.rt * a.tile_rows); };
  auto tiles_of = [&](int rows) { return rows > kWRows ? 2 : 1; };
  // halves of a tile of keys that hold any: the tree's own rows lie in the first
  auto halves_of = [&](const Walk& w, int j) {
    return j >= w.seq.cached || w.seq.hi - ((w.seq.lo >> kBTileLog) + j) * kBTile <= kBTile / 2 ? 1 : 2;
  };

  if (warp >= kBSoftWarps && warp < kBSoftWarps + kBDeqWarps) {
    // ------------------------------------------------------------------ dequant: four warps a side, 32 keys each
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    const int side = (warp - kBSoftWarps) >> 2, dw = warp & 3;
    const uint32_t low = side == 0 ? kBPow2Low : kBPow2LowQV;
    const int ch = lane % NCH;
    constexpr int kStep = 32 / NCH;
    const int sub = lane / NCH;
    const uint8_t* ring = smem + C::kOffRaw + side * C::kSlots * C::kRaw + (dw & 1) * 2 * L::kGranuleBytes;
    const uint32_t rfull = raw_full + side * 24, rempty = raw_empty + side * 24;
    const uint32_t full = side == 0 ? kfull : vfull, empty = side == 0 ? kempty : vempty;
    uint32_t to[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int pc = piece_of_word<D>(ch * 4 + k);
      to[k] = smem_u32(smem) + side * C::kOffV + (pc >> 3) * (kBTile * 128) + (dw * 32 + sub) * 128 +
              (((pc & 7) ^ (sub & 7)) << 4);
    }
    const uint8_t* codes0 = ring + sub * L::kRow + ch * 16;
    const uint8_t* par0 = ring + (lane >> 4) * L::kGranuleBytes + L::kCodes + (lane & 15) * L::kGroups * 4;
    uint32_t it = 0, half = static_cast<uint32_t>(dw >> 1);  // the warp's next half of a tile: every other one
    for (Walk w(a, range); w.valid(); w.next(a)) {
      const __nv_bfloat16* own_src = (side == 0 ? a.k_new : a.v_new) + static_cast<int64_t>(w.b) * a.G * a.new_stride + w.head * D;
      if (w.j1 > w.seq.cached && dw * 32 + lane < a.G)  // the piece ends with its own rows
#pragma unroll
        for (int x = 0; x < D; x += 64) prefetch_l1(own_src + (dw * 32 + lane) * a.new_stride + x);
      const int at = (w.seq.lo & ~(kBTile - 1)) + dw * 32 + lane;
      const int seen_lo = w.seq.lo - at, seen_hi = w.seq.hi - at;
#pragma unroll 1
      for (int j = w.j0; j < w.j1; ++j, ++it) {
        const uint32_t buf = it & 1u, par = ((it >> 1) & 1u) ^ 1u, tile = buf * C::kTileBytes;
        WideInfo* info = info_of(it);
        float* inf = reinterpret_cast<float*>(info->key + dw * 32) + side;
        if (j < w.seq.cached) {
          const uint32_t slot = half % C::kSlots;
          wait_on(rfull + 8 * slot, (half / C::kSlots) & 1u, abort_flag, a.err);
          const bool in = ((came_s[side * 3 + slot] >> (2 * (dw & 1) + (lane >> 4))) & 1u) && j * kBTile >= seen_lo && j * kBTile < seen_hi;
          const uint32_t raw = slot * C::kRaw;
          uint4 c[NCH];
#pragma unroll
          for (int i = 0; i < NCH; ++i)  // every load before the first store
            c[i] = *reinterpret_cast<const uint4*>(
                codes0 + raw + (D == 128 ? (i >> 1) * L::kGranuleBytes + (i & 1) * 8 * L::kRow : i * L::kGranuleBytes));
          uint32_t pr[2] = {0u, 0u}, po[2] = {0u, 0u};
          if (in) {
            pr[0] = *reinterpret_cast<const uint32_t*>(par0 + raw);
            if (L::kGroups == 2) pr[1] = *reinterpret_cast<const uint32_t*>(par0 + raw + 4);
          }
          // (a value row that is not finite counts as zeros, with a factor of NaN: only rows that see it become NaN)
          const bool odd = side == 1 && (pair_not_finite(pr[0]) || (L::kGroups == 2 && pair_not_finite(pr[1])));
          if (odd) pr[0] = pr[1] = 0u;
          // one power of two for the 32 keys, if they lie close enough
          const float largest = row_largest<L::kGroups>(pr), own = pow2_of(largest, low);
          const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(own));
          const uint32_t least = __reduce_min_sync(0xffffffffu, largest > 0.f ? __float_as_uint(own) : top);
          const bool mixed = __any_sync(0xffffffffu, odd) || __uint_as_float(least) * kWSpread < __uint_as_float(top);
          const float p2 = mixed ? own : __uint_as_float(top), inv = pow2_inverse(p2) * 0.0078125f;
#pragma unroll
          for (int g = 0; g < L::kGroups; ++g) {
            const float2 p = __bfloat1622float2(as_bf162(pr[g]));
            const __half2 h = __floats2half2_rn(p.x * inv * 16777216.f, p.y * inv);
            po[g] = *reinterpret_cast<const uint32_t*>(&h);
          }
          const float f = odd ? __uint_as_float(0x7fffffffu) : p2 * 128.f;
          uint32_t sb_bits[NCH];
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            const uint32_t w0 = __shfl_sync(0xffffffffu, po[0], sub + i * kStep);
            const uint32_t w1 = L::kGroups == 2 ? __shfl_sync(0xffffffffu, po[1], sub + i * kStep) : w0;
            sb_bits[i] = ch >= 2 ? w1 : w0;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(rempty + 8 * slot);
          half += 2;
          wait_on(empty + 8 * buf, par, abort_flag, a.err);
          inf[2 * lane] = side == 0 || in ? f : -1.f;
          const uint32_t there = __ballot_sync(0xffffffffu, in);
          if (lane == 0) {
            (side == 0 ? info->k : info->v)[dw] = f;
            (side == 0 ? info->mixed_k : info->mixed_v)[dw] = mixed ? 1u : 0u;
            if (side == 1) info->there[dw] = there;
          }
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            const __half2 sb = *reinterpret_cast<const __half2*>(&sb_bits[i]);
            const __half2 s24 = __low2half2(sb), b = __high2half2(sb);
            const __half2 s20 = __hmul2(s24, __float2half2_rn(0.0625f));
            const uint32_t cw[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) st_shared_v4(to[k] + tile + i * kStep * 128, dequant_word(cw[k], s24, s20, b));
          }
        } else {
          // the sequence's own rows: their powers of two, then (read again) the operands. (Loops, here and below: code that
          // runs once an item is fetched for it, and straight lines of it take longer than their work.)
          const uint32_t kOdd = 0x7fffffffu;  // a row that is not finite: values as for cached rows, keys become NaN
          float most = 0.f, least = 3e38f;
          wait_on(empty + 8 * buf, par, abort_flag, a.err);
#pragma unroll 1
          for (int i = 0; i < NCH; ++i) {
            const int t = sub + i * kStep, key = dw * 32 + t;
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key < a.G) m = max(m, max_abs8(__ldg(reinterpret_cast<const uint4*>(own_src + key * a.new_stride + ch * 32 + 8 * k))));
#pragma unroll
            for (int x = 1; x < NCH; x <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, x));
            const float own = m >= kBInfinity ? __uint_as_float(kOdd) : pow2_of(__uint_as_float(m), low);
            if (m >= kBInfinity) {
              if (side == 1) least = 0.f;
            } else if (m > 0) {
              least = fminf(least, own);
              most = fmaxf(most, own);
            }
            if (ch == 0) inf[2 * t] = own;
          }
          most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
          least = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(least)));
          if (most == 0.f) most = 1.f;
          const bool mixed = least * kWSpread < most;
          __syncwarp();
#pragma unroll 1
          for (int i = 0; i < NCH; ++i) {
            const int t = sub + i * kStep, key = dw * 32 + t;
            const float own = inf[2 * t], p2 = mixed ? own : most;
            const bool odd = __float_as_uint(own) == kOdd;
            const uint32_t none = side == 0 && odd ? 0x7fff7fffu : 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint4 u = make_uint4(none, none, none, none);
              if (key < a.G && !odd)
                u = convert_word(__ldg(reinterpret_cast<const uint4*>(own_src + key * a.new_stride + ch * 32 + 8 * k)), pow2_inverse(p2));
              st_shared_v4(to[k] + tile + i * kStep * 128, u);
            }
            __syncwarp();
            if (ch == 0) inf[2 * t] = side == 0 ? (odd ? 1.f : p2) : (key < a.G ? (odd ? own : p2) : -1.f);
          }
          if (lane == 0) {
            (side == 0 ? info->k : info->v)[dw] = most;
            (side == 0 ? info->mixed_k : info->mixed_v)[dw] = mixed ? 1u : 0u;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full + 8 * buf);
      }
    }
  } else if (warp == kBMmaWarp || warp == kBMmaWarp + 1) {
    // ------------------------------------------------------------------ MMA issuers: S, and O
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (elect_one()) {
      uint32_t it = 0, done[2] = {0u, 0u}, pieces[2] = {0u, 0u};  // tiles of keys; a row tile's products, its items
      if (warp == kBMmaWarp) {
        constexpr uint32_t kFmt = (1u << 4) | (static_cast<uint32_t>(64 >> 3) << 17) | (8u << 24);  // f32 <- f16, M = 128, N = 64
        const uint64_t kd = desc_kmajor_sw128(smem_u32(smem)), qd = desc_kmajor_sw128(smem_u32(smem + C::kOffQ));
        const uint32_t hi = static_cast<uint32_t>(kd >> 32), k_lo = static_cast<uint32_t>(kd), q_lo = static_cast<uint32_t>(qd);
        for (Walk w(a, range); w.valid(); w.next(a)) {
          const int nt = tiles_of(rows_of(w));
          for (int t = 0; t < nt; ++t) {
            wait_on(qfull + 8 * t, pieces[t] & 1u, abort_flag, a.err);
            ++pieces[t];
          }
#pragma unroll 1
          for (int j = w.j0; j < w.j1; ++j, ++it) {
            const uint32_t buf = it & 1u, k = k_lo + buf * (C::kTileBytes / 16);
            wait_on(kfull + 8 * buf, (it >> 1) & 1u, abort_flag, a.err);
            const int nh = halves_of(w, j);
#pragma unroll 1
            for (int x = 0; x < nh * nt; ++x) {
              const int t = nt == 2 ? x & 1 : 0;
              const uint32_t n = done[t]++, at = 2 * t + (n & 1u);
              if (n > 1) wait_on(odone + 8 * at, ((n >> 1) - 1) & 1u, abort_flag, a.err);  // P is read
              tc_fence_after();
              const uint32_t q = q_lo + t * (C::kTileBytes / 16), d = tmem + at * 64, kh = k + (nt == 2 ? x >> 1 : x) * (64 * 128 / 16);
              mma_lean<true>(d, q, kh, hi, hi, kFmt);
#pragma unroll
              for (int s = 1; s < D / 16; ++s) {
                const uint32_t o = (s >> 2) * (kBTile * 128 / 16) + 2 * (s & 3);
                mma_lean<false>(d, q + o, kh + o, hi, hi, kFmt);
              }
              mma_commit(sfull + 8 * at);
            }
            mma_commit(kempty + 8 * buf);
          }
        }
      } else {
        constexpr uint32_t kFmt = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (8u << 24);
        const uint64_t vd = desc_keys_sw128(smem_u32(smem + C::kOffV));
        const uint32_t hi = static_cast<uint32_t>(vd >> 32), v_lo = static_cast<uint32_t>(vd);
        for (Walk w(a, range); w.valid(); w.next(a)) {
          const int nt = tiles_of(rows_of(w));
#pragma unroll 1
          for (int j = w.j0; j < w.j1; ++j, ++it) {
            const uint32_t buf = it & 1u, v = v_lo + buf * (C::kTileBytes / 16);
            wait_on(vfull + 8 * buf, (it >> 1) & 1u, abort_flag, a.err);
            const int nh = halves_of(w, j);
#pragma unroll 1
            for (int x = 0; x < nh * nt; ++x) {
              const int t = nt == 2 ? x & 1 : 0, h = nt == 2 ? x >> 1 : x;
              const uint32_t n = done[t]++, at = 2 * t + (n & 1u);
              wait_on(pfull + 8 * at, (n >> 1) & 1u, abort_flag, a.err);
              tc_fence_after();
              const uint32_t p = tmem + at * 64, d = tmem + 256 + t * kWRows, vh = v + h * (4 * 128);
              if (j > w.j0 || h > 0)
                mma_tmem<false>(d, p, vh, hi, kFmt);
              else
                mma_tmem<true>(d, p, vh, hi, kFmt);
#pragma unroll
              for (int s = 1; s < 4; ++s) mma_tmem<false>(d, p + 8 * s, vh + 128 * s, hi, kFmt);
              mma_commit(odone + 8 * at);
            }
            mma_commit(vempty + 8 * buf);
          }
        }
      }
      if (*abort_flag != 0) {  // the MMAs in flight end before the CTA leaves
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp >= kBCopyWarp) {
    // ------------------------------------------------------------------ copies of one side, 64 keys at a time
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    const int side = warp - kBCopyWarp;
    const int granules = (1 << a.page_shift) / kKvGranule, run = min(granules, 4);
    const uint32_t rfull = raw_full + side * 24, rempty = raw_empty + side * 24;
    uint32_t half = 0;
    for (Walk w(a, range); w.valid(); w.next(a)) {
      const int last = min(w.j1, w.seq.cached);
      for (int j0 = w.j0; j0 < last; j0 += 4) {  // pages of four tiles at a time: 32 granules, one a lane
        const int g0 = ((w.seq.lo >> kBTileLog) + j0) * (kBTile / kKvGranule) + lane;
        const int key = g0 * kKvGranule;
        int page = -1;
        if (j0 + lane / 8 < last && key < w.seq.hi && key + kKvGranule > w.seq.lo) {
          page = __ldg(a.table + static_cast<int64_t>(w.b) * a.width + (key >> a.page_shift));
          if (page < 0 || page >= a.num_pages) {
            atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_BAD_INDEX));
            page = -1;
          }
        }
        const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
        for (int h = 0; h < 2 * (min(j0 + 4, last) - j0); ++h, ++half) {
          const uint32_t got = (have >> (4 * h)) & 0xfu, slot = half % C::kSlots;
          wait_on(rempty + 8 * slot, ((half / C::kSlots) & 1u) ^ 1u, abort_flag, a.err);
          if (lane == 0) {
            came_s[side * 3 + slot] = got;
            mbar_arrive_expect_tx(rfull + 8 * slot, static_cast<uint32_t>(__popc(got)) * L::kGranuleBytes);
          }
          __syncwarp();
          // the granules of a run that lies together in a page, copied by the lane of the first that came
          const int g = lane & 3, first = g & ~(run - 1);
          const uint32_t mine = (got >> first) & ((1u << run) - 1u);
          if (lane / 4 == h && mine != 0u && g == first + __ffs(mine) - 1)
            bulk_load(smem_u32(smem + C::kOffRaw + (side * C::kSlots + slot) * C::kRaw + g * L::kGranuleBytes),
                      a.cache + (((static_cast<int64_t>(page) * a.Hkv + w.head) * 2 + side) * granules +
                                 (g0 & (granules - 1))) *
                                    static_cast<int64_t>(L::kGranuleBytes),
                      static_cast<uint32_t>(__popc(mine)) * L::kGranuleBytes, rfull + 8 * slot);
          __syncwarp();
        }
      }
    }
  } else if (warp < kBSoftWarps) {
    // ------------------------------------------------------------------ softmax: a thread a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    const int t = warp >> 2, in_tile = threadIdx.x & (kWRows - 1);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * kBTile, to = tmem + lanes + 256 + t * kWRows;
    float* qs_of = reinterpret_cast<float*>(smem + C::kOffQs) + t * kWRows;
    struct Row {             // of the thread, in its item
      int r, tok, head_row;  // its place among the item's rows, its token and its query head
      bool exists, there;
      uint64_t line;         // the own rows that it sees
      int row_lo, all_lo;    // its first cached key; the last of the warp's rows' first
      float qs;              // what its scores are multiplied by
    };
    // An item's rows, as far as they are this row tile's: lines of ancestors, and Q over each row's own power of two; a row
    // that is not finite becomes NaN, one that is not there zeros. (Every S of the item before is done.)
    auto load_item = [&](const Walk& w, Row& row) {
      const int nrows = rows_of(w), nt = tiles_of(nrows), per = nt == 1 ? nrows : (nrows + 1) / 2;
      constexpr int kPieces = D / 8, kAt = 32 / kPieces;   // lanes a row, rows at a time
      auto place = [&](int in, int& r, int& tok, int& head_row) {
        r = t * per + in;
        const bool exists = t < nt && in < per && r < nrows;
        const int rr = w.rt * a.tile_rows + (exists ? r : 0);
        tok = row_token(a, rr);
        head_row = w.head * a.R + rr - tok * a.R;
        return exists;
      };
      int parent[2] = {-2, -2};
      if ((warp & 3) == 0)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (lane + 32 * i < a.G) parent[i] = __ldg(a.parents + static_cast<int64_t>(w.b) * a.G + lane + 32 * i);
      if ((warp & 3) == 0) {
        bool bad;
        const TreeLines tree = tree_lines(parent, a.G, bad);
        if (bad) atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_BAD_INDEX));
        tree_line[t * kTreeRows + lane] = tree.line[0];
        tree_line[t * kTreeRows + lane + 32] = tree.line[1];
      }
      asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + t), "n"(kWRows) : "memory");
      if (t >= nt) return;
      const int pc = piece_of_word<D>(lane % kPieces);
      uint8_t* q_to = smem + C::kOffQ + t * C::kTileBytes + (pc >> 3) * (kWRows * 128);
      const float lift = a.scale_log2 < 0.f ? -kBLiftQ : kBLiftQ;
#pragma unroll 1
      for (int i0 = 0; i0 < kPieces; i0 += 4) {  // (rolled: code that runs once an item is fetched for it)
        uint4 v[4];
        bool there[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int r, tok, head_row;
          there[i] = place((warp & 3) * 32 + (i0 + i) * kAt + lane / kPieces, r, tok, head_row) && tree_line[t * kTreeRows + tok] != 0ull;
          v[i] = there[i] ? __ldg(reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(w.b) * a.G + tok) * a.q_stride + head_row * D) +
                                  lane % kPieces)
                          : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int in = (warp & 3) * 32 + (i0 + i) * kAt + lane / kPieces;
          uint32_t m = max_abs8(v[i]);
#pragma unroll
          for (int x = 1; x < kPieces; x <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, x));
          const float own = pow2_of(__uint_as_float(m), kBPow2LowQV);
          const uint4 u = m < kBInfinity ? convert_word(v[i], lift * pow2_inverse(own))
                                         : make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
          *reinterpret_cast<uint4*>(q_to + in * 128 + (((pc & 7) ^ (in & 7)) << 4)) = u;
          if (lane % kPieces == 0) qs_of[in] = own * (1.f / kBLiftQ) * fabsf(a.scale_log2);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull + 8 * t);
      row.exists = place(in_tile, row.r, row.tok, row.head_row);
      row.line = row.exists ? tree_line[t * kTreeRows + row.tok] : 0ull;
      row.there = row.line != 0ull;
      const int pos = w.seq.L + __popcll(row.line) - 1;
      row.row_lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      if (a.window > 0)
        for (int n = __popcll(row.line); n > a.window; --n) row.line &= row.line - 1ull;
      row.all_lo = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<uint32_t>(row.there ? row.row_lo : 0)));
      row.qs = qs_of[in_tile];
      __syncwarp();
    };
    uint32_t it = 0, n = 0;  // tiles of keys; this row tile's halves of them
    Row row, me;
    Walk next(a, range), w = next;
    if (threadIdx.x == 0) {
      int2 e = make_int2(-1, 0);
      if (next.valid() && next.j0 > 0 && next.j1 == next.seq.tiles)
        e = make_int2((next.b * a.Hkv + next.head) * a.row_tiles + next.rt,
                      BlockParts(range.line, next.start, kWSetup, next.seq.tiles).c0);
      wa.entry[blockIdx.x] = e;
    }
    float ref = 0.f, l = 0.f;  // minus the reference; the sum
    bool mine = false;         // the item before had rows of this tile
    for (;;) {
      if (next.valid()) load_item(next, row);  // (its scores are computed while the item before is finished)
      if (mine) {
        // ---- the result of the item before, or this range's part of it
        wait_on(odone + 16 * t + 8 * ((n - 1) & 1u), ((n - 1) >> 1) & 1u, abort_flag, a.err);
        __syncwarp();
        tc_fence_after();
        const bool complete = w.j0 == 0 && w.j1 == w.seq.tiles;
        if (!me.there) l = 0.f;  // (whatever a row that is not there holds)
        const float g = l == 0.f ? 0.f : (complete ? kBSumUnit / l : 1.f);
        const int64_t slot = (static_cast<int64_t>(blockIdx.x) * 2 + (w.j0 > 0 ? 0 : 1)) * (2 * kWRows) + me.r;
        __nv_bfloat16* out = a.out + ((static_cast<int64_t>(w.b) * a.G + me.tok) * a.Hq + me.head_row) * D;
        float* part = a.part_o + slot * D;
        if (me.exists && !complete) a.part_ml[slot] = make_float2(ref != kBUnseen && me.there ? -ref : -INFINITY, l);
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t raw[16];
          float o[16];
          tmem_ld16(to + c, raw);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = g != 0.f ? __uint_as_float(raw[i]) * g : 0.f;  // (O of a row that saw nothing is not looked at)
          if (complete && me.exists) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // positions hold channels 0, 4, 1, 5, 2, 6, 3, 7 of a word
              uint32_t u[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int from = 8 * k + (i < 2 ? 4 * i : 4 * (i - 2) + 1);
                const __nv_bfloat162 v = __floats2bfloat162_rn(o[from], o[from + 2]);
                u[i] = *reinterpret_cast<const uint32_t*>(&v);
              }
              *reinterpret_cast<uint4*>(out + word_of_piece<D>(c / 8 + k) * 8) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          } else if (me.exists) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              __stcg(reinterpret_cast<float4*>(part + c + i), make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
          }
        }
        __syncwarp();
        tc_fence_before();
      }
      if (!next.valid()) break;
      w = next;
      me = row;
      next.next(a);
      mine = t < tiles_of(rows_of(w));
      if (next.valid()) {  // its queries and parents are on their way meanwhile
        const int rows = rows_of(next), tiles = tiles_of(rows), r = t * (tiles == 1 ? rows : (rows + 1) / 2) + in_tile;
        const int rr = next.rt * a.tile_rows + min(r, rows - 1), tok = row_token(a, rr);
        const __nv_bfloat16* q = a.q + (static_cast<int64_t>(next.b) * a.G + tok) * a.q_stride + (next.head * a.R + rr - tok * a.R) * D;
#pragma unroll
        for (int x = 0; x < D; x += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + x));
        if (in_tile < a.G) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.parents + static_cast<int64_t>(next.b) * a.G + in_tile));
      }
      if (!mine) {
        it += static_cast<uint32_t>(w.j1 - w.j0);
        continue;
      }
      ref = me.there ? kBUnseen : kBPadding;
      l = 0.f;
#pragma unroll 1
      for (int j = w.j0; j < w.j1; ++j, ++it) {
        const bool own = j >= w.seq.cached;
        const int key0 = own ? w.seq.L : ((w.seq.lo >> kBTileLog) + j) * kBTile;
        const int nh = halves_of(w, j);
#pragma unroll 1
        for (int h = 0; h < nh; ++h, ++n) {
          const uint32_t at = n & 1u;
          // (the scores first: where items of one row tile came before, only they tell the second's warps how far the
          // values' barrier has come)
          wait_on(sfull + 16 * t + 8 * at, (n >> 1) & 1u, abort_flag, a.err);
          if (h == 0) wait_on(vfull + 8 * (it & 1u), (it >> 1) & 1u, abort_flag, a.err);
          __syncwarp();
          tc_fence_after();
          float x[64];  // the half's scores, then numbers
          tmem_ld32(ts + 64 * at, reinterpret_cast<float(&)[32]>(x[0]));
          tmem_ld32(ts + 64 * at + 32, reinterpret_cast<float(&)[32]>(x[32]));
          const WideInfo* info = info_of(it);
          const uint2 th = *reinterpret_cast<const uint2*>(info->there + 2 * h), mk = *reinterpret_cast<const uint2*>(info->mixed_k + 2 * h),
                      mv = *reinterpret_cast<const uint2*>(info->mixed_v + 2 * h);
          const float2 k2 = *reinterpret_cast<const float2*>(info->k + 2 * h), v2 = *reinterpret_cast<const float2*>(info->v + 2 * h);
          const bool mixed = (mk.x | mk.y | mv.x | mv.y) != 0u;
          const bool plain = !own && !mixed && key0 >= me.all_lo && (th.x & th.y) == ~0u;
          const float fk[2] = {k2.x * me.qs, k2.y * me.qs}, fv[2] = {v2.x, v2.y};
          auto log_of = [](float f) { return static_cast<float>(static_cast<int>(__float_as_uint(f) >> 23) - 127); };
          // raises the reference where the half's largest number passes it, in straight-line code; O and the sum follow
          auto raise = [&](float most) {
            if (!__any_sync(0xffffffffu, most + ref > kBSlack)) return;
            const float up = kBLift - most;
            float shrink = 1.f;
            if (ref != kBPadding && most > -INFINITY && most + ref > kBSlack && up < ref) {
              shrink = ref == kBUnseen ? 0.f : ex2_approx(up - ref);
              ref = up;
              l *= shrink;
            }
            if (j == w.j0 && h == 0) return;
            wait_on(odone + 16 * t + 8 * (at ^ 1u), ((n - 1) >> 1) & 1u, abort_flag, a.err);  // the half before is in O
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(to + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * shrink);
              tmem_st16(to + c, o);
            }
            tmem_st_wait();
          };
          // which of the half's keys the row sees
          uint32_t seen[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int from = me.row_lo - key0 - 64 * h - 32 * c;  // the group's first key after the window's start
            seen[c] = own ? static_cast<uint32_t>(me.line >> (32 * c))
                          : (from >= 32 || !me.there ? 0u : (c == 0 ? th.x : th.y) & (from > 0 ? ~0u << from : ~0u));
          }
          // probabilities times the values' factors, over S, and their sum without those
          auto weigh = [&]() {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float2 sum = make_float2(0.f, 0.f);
              uint32_t p[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 y = __fadd2_rn(make_float2(x[32 * c + 2 * i], x[32 * c + 2 * i + 1]), make_float2(ref, ref));
                const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                sum = __fadd2_rn(sum, e);
                const __half2 h2 = __floats2half2_rn(e.x, e.y);
                p[i] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              l = fmaf(sum.x + sum.y, pow2_inverse(fv[c]) * kBSumUnit, l);
              tmem_st16(ts + 64 * at + 16 * c, p);
            }
          };
          tmem_ld_wait();
          if (plain) {
            // (The reference is subtracted from rounded numbers, among them the maximum it was set to: inside the FMA, the
            // largest of very large scores could pass any slack by its own rounding.)
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float vlog = log_of(fv[c]);
#pragma unroll
              for (int i = 32 * c; i < 32 * c + 32; i += 2) {
                const float2 z = __ffma2_rn(make_float2(x[i], x[i + 1]), make_float2(fk[c], fk[c]), make_float2(vlog, vlog));
                x[i] = z.x;
                x[i + 1] = z.y;
                m0 = fmaxf(m0, z.x);
                m1 = fmaxf(m1, z.y);
              }
            }
            raise(fmaxf(m0, m1));
            weigh();
          } else if (!mixed) {
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float vlog = log_of(fv[c]);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 z = __ffma2_rn(make_float2(x[32 * c + i], x[32 * c + i + 1]), make_float2(fk[c], fk[c]), make_float2(vlog, vlog));
                x[32 * c + i] = (seen[c] & (1u << i)) != 0u ? z.x : -INFINITY;
                x[32 * c + i + 1] = (seen[c] & (2u << i)) != 0u ? z.y : -INFINITY;
                m0 = fmaxf(m0, x[32 * c + i]);
                m1 = fmaxf(m1, x[32 * c + i + 1]);
              }
            }
            raise(fmaxf(m0, m1));
            weigh();
          } else {
            // rows that lie far apart: a factor a key
            // (eight keys at a time: the numbers are made twice, from S, of which P takes the first half behind it)
            auto numbers = [&](int i0, float (&z)[8]) {
              tmem_ld8(ts + 64 * at + i0, z);
              const uint32_t bits = (i0 < 32 ? seen[0] : seen[1]) >> (i0 & 31);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 k = info->key[64 * h + i0 + i];  // (the values' may be NaN)
                z[i] = (bits & (1u << i)) != 0u ? fmaf(z[i], k.x * me.qs, fmaf(k.y, 0.f, log_of(k.y))) : -INFINITY;
              }
            };
            float most = -INFINITY;
#pragma unroll 1
            for (int i0 = 0; i0 < 64; i0 += 8) {
              float z[8];
              numbers(i0, z);
#pragma unroll
              for (int i = 0; i < 8; ++i) most = fmaxf(most, z[i]);
            }
            raise(most);
#pragma unroll 1
            for (int i0 = 0; i0 < 64; i0 += 8) {
              float z[8], sum = 0.f;
              uint32_t p[4];
              numbers(i0, z);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float e0 = ex2_approx(z[2 * i] + ref), e1 = ex2_approx(z[2 * i + 1] + ref);
                const float4 k = *reinterpret_cast<const float4*>(info->key + 64 * h + i0 + 2 * i);
                sum = fmaf(e0, pow2_inverse(k.y), fmaf(e1, pow2_inverse(k.w), sum));
                const __half2 h2 = __floats2half2_rn(e0, e1);
                p[i] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              l = fmaf(sum, kBSumUnit, l);
              tmem_st4(ts + 64 * at + i0 / 2, p);
            }
          }
          __syncwarp();
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull + 16 * t + 8 * at);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kBMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of items that several ranges share: a warp a row, eight rows a CTA.
constexpr int kJoinRows = 8, kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv4_wide_join_kernel(const WideArgs wa) {
  const BlockArgs& a = wa.a;
  constexpr int kCtas = 2 * kWRows / kJoinRows, kE = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int range = static_cast<int>(blockIdx.x) / kCtas;
  const int2 e = __ldcg(wa.entry + range);
  if (e.x < 0) return;
  const int rt = e.x % a.row_tiles, bh = e.x / a.row_tiles, b = bh / a.Hkv, head = bh - b * a.Hkv;
  const int n = range - e.y + 1, nrows = min(a.tile_rows, a.rows - rt * a.tile_rows);
  const int r = (static_cast<int>(blockIdx.x) - range * kCtas) * kJoinRows + warp;
  if (r >= nrows) return;
  auto slot = [&](int p) { return (static_cast<int64_t>(e.y + p) * 2 + (p == 0 ? 1 : 0)) * (2 * kWRows) + r; };
  float top = -INFINITY, sum = 0.f, acc[kE] = {};
  for (int p0 = 0; p0 < n; p0 += 8) {  // eight parts at a time, asked for before their weights are known
    const float2 ml = lane < 8 && p0 + lane < n ? __ldcg(a.part_ml + slot(p0 + lane)) : make_float2(-INFINITY, 0.f);
    float v[8][kE];
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
      for (int x = 0; x < kE; x += 2) {
        const float2 u = p0 + p < n ? __ldcg(reinterpret_cast<const float2*>(a.part_o + slot(p0 + p) * D + lane * kE + x)) : make_float2(0.f, 0.f);
        v[p][x] = u.x;
        v[p][x + 1] = u.y;
      }
    float most = fmaxf(top, ml.x);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
    const float shrink = top == -INFINITY ? 0.f : ex2_approx(top - most), f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - most);
    top = most;
    sum = fmaf(f, ml.y, sum * shrink);
#pragma unroll
    for (int x = 0; x < kE; ++x) acc[x] *= shrink;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float weight = __shfl_sync(0xffffffffu, f, p);
      if (weight != 0.f)  // (0: nothing of the row there)
#pragma unroll
        for (int x = 0; x < kE; ++x) acc[x] = fmaf(weight, v[p][x], acc[x]);
    }
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  const float inv = sum == 0.f ? 0.f : kBSumUnit / sum;
  const int rr = rt * a.tile_rows + r, t = row_token(a, rr);
  __nv_bfloat16* out = a.out + ((static_cast<int64_t>(b) * a.G + t) * a.Hq + head * a.R + rr - t * a.R) * D;
#pragma unroll
  for (int x = 0; x < kE; ++x) {
    const int p = lane * kE + x;
    out[word_of_piece<D>(p >> 3) * 8 + ((p & 7) >> 1) + 4 * (p & 1)] = __float2bfloat16_rn(inv != 0.f ? acc[x] * inv : 0.f);
  }
}

struct WidePlan {
  int row_tiles, tile_rows, ctas;
  int64_t items;
  size_t ml, entry, total;
};
WidePlan wide_plan(int B, int G, int Hq, int Hkv, int D, int64_t max_ctx, int sms) {
  WidePlan p;
  const int rows = G * (Hq / Hkv);
  p.row_tiles = (rows + 2 * kWRows - 1) / (2 * kWRows);
  p.tile_rows = (rows + p.row_tiles - 1) / p.row_tiles;
  p.items = static_cast<int64_t>(B) * Hkv * p.row_tiles;
  p.ctas = static_cast<int>(std::min<int64_t>(sms, p.items * ((max_ctx + kBTile - 1) / kBTile + 1)));
  const size_t slots = static_cast<size_t>(p.ctas) * 2 * (2 * kWRows);
  p.ml = slots * D * sizeof(float);
  p.entry = p.ml + slots * sizeof(float2);
  p.total = p.entry + static_cast<size_t>(p.ctas) * sizeof(int2);
  return p;
}

template <int D>
int launch_wide_t(const WideArgs& a, const WidePlan& p, cudaStream_t st) {
  using C = WideCfg<D>;
  static_assert(C::kSmem <= 232448, "shared memory");
  static_assert(kBSoft * C::kSoftRegs + (kBThreads - kBSoft) * C::kOtherRegs <= kBThreads * 96, "registers");
  static unsigned done = 0;
  if (!ensure_smem_attr(kv4_wide_kernel<D>, C::kSmem, &done)) return fail(DFLASH2_ERR_CUDA, "cudaFuncSetAttribute failed (attention)");
  cudaError_t e = launch_pdl(kv4_wide_kernel<D>, dim3(static_cast<unsigned>(p.ctas)), dim3(kBThreads), C::kSmem, st, nullptr, 0, a);
  if (e == cudaSuccess)
    e = launch_pdl(kv4_wide_join_kernel<D>, dim3(static_cast<unsigned>(p.ctas * (2 * kWRows / kJoinRows))), dim3(kJoinThreads), 0, st,
                   nullptr, 0, a);
  return e == cudaSuccess ? DFLASH2_OK : fail(DFLASH2_ERR_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
}

}  // namespace

bool kv4_wide_eligible(int B, int G, int Hq, int Hkv) {
  return G * (Hq / Hkv) > kWideRows && static_cast<int64_t>(B) * Hkv * (G * (Hq / Hkv) / (2 * kWRows) + 1) < (1 << 26);
}
size_t kv4_wide_workspace(int B, int G, int Hq, int Hkv, int D, int page_size, int max_pages, int sms) {
  return wide_plan(B, G, Hq, Hkv, D, static_cast<int64_t>(max_pages) * page_size, sms).total;
}

int launch_kv4_wide(const Kv4Attention& r, cudaStream_t st) {
  const WidePlan p = wide_plan(r.B, r.G, r.Hq, r.Hkv, r.D, static_cast<int64_t>(r.max_pages) * r.page_size, sm_count());
  WideArgs w{};
  BlockArgs& a = w.a;
  if (!block_args(r, p.ctas, p.row_tiles, p.tile_rows, a)) return fail(DFLASH2_ERR_CUDA, "no device error word");
  uint8_t* ws = static_cast<uint8_t*>(r.workspace);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + p.ml);
  w.entry = reinterpret_cast<int2*>(ws + p.entry);
  return r.D == 64 ? launch_wide_t<64>(w, p, st) : launch_wide_t<128>(w, p, st);
}

}  // namespace dfl
