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
// Ranges of the line leave partial results in the workspace; which ranges share an item is written beside them by the
// one that ends it, and a second kernel joins them, a warp a row. (So no CTA waits for another.)
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
  static constexpr int kOffBar = kOffLine + 2 * kTreeRows * 8;
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

__device__ __forceinline__ void tmem_ld32(uint32_t t, float (&x)[32]) {
  tmem_ld_32x32b_x32(t, reinterpret_cast<uint32_t(&)[32]>(x));
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const float (&x)[32]) {
  uint32_t a[16], b[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = __float_as_uint(x[i]);
    b[i] = __float_as_uint(x[16 + i]);
  }
  tmem_st16(t, a);
  tmem_st16(t + 16, b);
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
  int2* entry;  // [item] the ranges that share it
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
  const uint32_t sfull = bars + 64, pfull = bars + 80, odone = bars + 96, qfull = bars + 112;  // [2] each: row tiles
  const uint32_t raw_full = bars + 128, raw_empty = bars + 176;                            // [side][3]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 224);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* came_s = tmem_slot + 2;  // [side][3]: the granules that came

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull + 8 * i, kBDeqWarps / 2);
      mbar_init(vfull + 8 * i, kBDeqWarps / 2);
      mbar_init(kempty + 8 * i, 1);
      mbar_init(vempty + 8 * i, 1);
      mbar_init(sfull + 8 * i, 1);
      mbar_init(pfull + 8 * i, 4);
      mbar_init(odone + 8 * i, 1);
      mbar_init(qfull + 8 * i, 4);
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
  const uint32_t tmem = *tmem_slot;  // S (then P) of the row tiles at columns 0 and 128, O at 256 and 384
  pdl_trigger();
  pdl_wait();
  const BlockRange range = block_range(a, kWSetup, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
  // an item's rows: one tile of them, or two of equal size
  auto rows_of = [&](const Walk& w) { return min(a.tile_rows, a.rows - w.rt * a.tile_rows); };
  auto tiles_of = [&](int rows) { return rows > kWRows ? 2 : 1; };

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
          // the sequence's own rows
          wait_on(empty + 8 * buf, par, abort_flag, a.err);
#pragma unroll 1
          for (int i = 0; i < NCH; ++i) {
            const int t = sub + i * kStep, key = dw * 32 + t;
            float f = 0.f;
            uint4 u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] = make_uint4(0u, 0u, 0u, 0u);
            if (dw * 32 + i * kStep < a.G) {
              uint32_t m = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (key < a.G) u[k] = __ldg(reinterpret_cast<const uint4*>(own_src + key * a.new_stride + ch * 32 + 8 * k));
#pragma unroll
              for (int k = 0; k < 4; ++k) m = max(m, max_abs8(u[k]));
#pragma unroll
              for (int x = 1; x < NCH; x <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, x));
              const float p2 = pow2_of(__uint_as_float(m), low);
              const bool odd = side == 1 && m >= kBInfinity;
              f = odd ? __uint_as_float(0x7fffffffu) : p2;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                u[k] = odd ? make_uint4(0u, 0u, 0u, 0u) : convert_word(u[k], pow2_inverse(p2));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) st_shared_v4(to[k] + tile + i * kStep * 128, u[k]);
            if (ch == 0) inf[2 * t] = side == 0 || key < a.G ? f : -1.f;
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
    if (lane == 0) {
      uint32_t it = 0, done[2] = {0u, 0u}, pieces[2] = {0u, 0u};  // tiles of keys; a row tile's products, its items
      if (warp == kBMmaWarp) {
        constexpr uint32_t kFmt = (1u << 4) | (static_cast<uint32_t>(kBTile >> 3) << 17) | (8u << 24);  // f32 <- f16, M = 128
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
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
              if (done[t] > 0) wait_on(odone + 8 * t, (done[t] - 1) & 1u, abort_flag, a.err);  // P is read
              ++done[t];
              tc_fence_after();
              const uint32_t q = q_lo + t * (C::kTileBytes / 16), d = tmem + t * kBTile;
              mma_lean<true>(d, q, k, hi, hi, kFmt);
#pragma unroll
              for (int s = 1; s < D / 16; ++s) {
                const uint32_t o = (s >> 2) * (kBTile * 128 / 16) + 2 * (s & 3);
                mma_lean<false>(d, q + o, k + o, hi, hi, kFmt);
              }
              mma_commit(sfull + 8 * t);
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
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
              wait_on(pfull + 8 * t, done[t] & 1u, abort_flag, a.err);
              ++done[t];
              tc_fence_after();
              const uint32_t p = tmem + t * kBTile, d = tmem + 256 + t * kWRows;
              if (j > w.j0)
                mma_tmem<false>(d, p, v, hi, kFmt);
              else
                mma_tmem<true>(d, p, v, hi, kFmt);
#pragma unroll
              for (int s = 1; s < kBTile / 16; ++s) mma_tmem<false>(d, p + 8 * s, v + 128 * s, hi, kFmt);
              mma_commit(odone + 8 * t);
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
    uint32_t it = 0, done = 0, piece = 0;  // tiles of keys; this row tile's, and its items
    for (Walk w(a, range); w.valid(); w.next(a), ++piece) {
      const int nrows = rows_of(w), nt = tiles_of(nrows);
      const int per = nt == 1 ? nrows : (nrows + 1) / 2;     // rows a tile
      // the lines of ancestors: the first warp of each row tile, which alone need not wait for the other's
      if ((warp & 3) == 0) {
        int parent[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          parent[i] = lane + 32 * i < a.G ? __ldg(a.parents + static_cast<int64_t>(w.b) * a.G + lane + 32 * i) : -2;
        bool bad;
        const TreeLines tree = tree_lines(parent, a.G, bad);
        if (bad) atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_BAD_INDEX));
        tree_line[t * kTreeRows + lane] = tree.line[0];
        tree_line[t * kTreeRows + lane + 32] = tree.line[1];
      }
      asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + t), "n"(kWRows) : "memory");
      if (t < nt) {
        const int r = t * per + in_tile;                     // of the item's rows
        const bool exists = in_tile < per && r < nrows;
        const int rr = w.rt * a.tile_rows + (exists ? r : 0), tok = row_token(a, rr);
        uint64_t line = exists ? tree_line[t * kTreeRows + tok] : 0ull;
        const bool there = line != 0ull;
        const int pos = w.seq.L + __popcll(line) - 1;
        const int row_lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
        if (a.window > 0)
          for (int n = __popcll(line); n > a.window; --n) line &= line - 1ull;
        const int all_lo = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<uint32_t>(there ? row_lo : 0)));
        // ---- Q over the row's own power of two; a row that is not finite becomes NaN, one that is not there zeros
        float qs;
        {
          const __nv_bfloat16* q = a.q + (static_cast<int64_t>(w.b) * a.G + tok) * a.q_stride + (w.head * a.R + rr - tok * a.R) * D;
          uint32_t m = 0;
          if (there)
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) m = max(m, max_abs8(__ldg(reinterpret_cast<const uint4*>(q) + c)));
          const float own = pow2_of(__uint_as_float(m), kBPow2LowQV);
          qs = own * (1.f / kBLiftQ) * fabsf(a.scale_log2);
          const float by = (a.scale_log2 < 0.f ? -kBLiftQ : kBLiftQ) * pow2_inverse(own);
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (there) v = m < kBInfinity ? convert_word(__ldg(reinterpret_cast<const uint4*>(q) + c), by)
                                          : make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
            const int pc = piece_of_word<D>(c);
            *reinterpret_cast<uint4*>(smem + C::kOffQ + t * C::kTileBytes + (pc >> 3) * (kWRows * 128) + in_tile * 128 +
                                      (((pc & 7) ^ (in_tile & 7)) << 4)) = v;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(qfull + 8 * t);
        }
        float ref = there ? kBUnseen : kBPadding, l = 0.f;   // minus the reference; the sum
        // raises the reference where the tile's largest number passes it, in straight-line code; O and the sum follow
        auto raise = [&](float most, bool rescale) {
          const float next = kBLift - most;
          float shrink = 1.f;
          if (ref != kBPadding && most > -INFINITY && most + ref > kBSlack && next < ref) {
            shrink = ref == kBUnseen ? 0.f : ex2_approx(next - ref);
            ref = next;
            l *= shrink;
          }
          if (!rescale) return;
          tc_fence_after();  // (the product before is done: the scores came after it)
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(to + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= shrink;
            tmem_st32(to + c, o);
          }
          tmem_st_wait();
        };
#pragma unroll 1
        for (int j = w.j0; j < w.j1; ++j, ++it, ++done) {
          const uint32_t buf = it & 1u;
          // (the scores first: where items of one row tile came before, only they tell the second's warps how far the
          // values' barrier has come)
          wait_on(sfull + 8 * t, done & 1u, abort_flag, a.err);
          wait_on(vfull + 8 * buf, (it >> 1) & 1u, abort_flag, a.err);
          __syncwarp();
          tc_fence_after();
          const WideInfo* info = info_of(it);
          const bool own = j >= w.seq.cached;
          const int key0 = own ? w.seq.L : ((w.seq.lo >> kBTileLog) + j) * kBTile;
          bool plain = !own && key0 >= all_lo;
          if (plain) {
            const uint4 th = *reinterpret_cast<const uint4*>(info->there), mk = *reinterpret_cast<const uint4*>(info->mixed_k),
                        mv = *reinterpret_cast<const uint4*>(info->mixed_v);
            plain = (th.x & th.y & th.z & th.w) == ~0u && (mk.x | mk.y | mk.z | mk.w | mv.x | mv.y | mv.z | mv.w) == 0u;
          }
          float x[32];
          if (plain) {
            const float4 k4 = *reinterpret_cast<const float4*>(info->k), v4 = *reinterpret_cast<const float4*>(info->v);
            const float fk[4] = {k4.x * qs, k4.y * qs, k4.z * qs, k4.w * qs}, fv[4] = {v4.x, v4.y, v4.z, v4.w};
            float most = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              tmem_ld32(ts + 32 * c, x);
              tmem_ld_wait();
              float m0 = x[0], m1 = x[1];
#pragma unroll
              for (int i = 2; i < 32; i += 2) {
                m0 = fmaxf(m0, x[i]);
                m1 = fmaxf(m1, x[i + 1]);
              }
              const float vlog = static_cast<float>(static_cast<int>(__float_as_uint(fv[c]) >> 23) - 127);
              most = fmaxf(most, fmaf(fmaxf(m0, m1), fk[c], vlog));
            }
            if (__any_sync(0xffffffffu, most + ref > kBSlack)) raise(most, j > w.j0);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              tmem_ld32(ts + 32 * c, x);
              const float off = static_cast<float>(static_cast<int>(__float_as_uint(fv[c]) >> 23) - 127) + ref;
              tmem_ld_wait();
              float2 sum = make_float2(0.f, 0.f);
              uint32_t p[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 y = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(fk[c], fk[c]), make_float2(off, off));
                const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                sum = __fadd2_rn(sum, e);
                const __half2 h = __floats2half2_rn(e.x, e.y);
                p[i] = *reinterpret_cast<const uint32_t*>(&h);
              }
              l = fmaf(sum.x + sum.y, pow2_inverse(fv[c]) * kBSumUnit, l);
              tmem_st16(ts + 16 * c, p);
            }
          } else {
            // masks, and a factor a key
            float most = -INFINITY;
            auto seen_of = [&](int c) {
              if (own) return c < 2 ? static_cast<uint32_t>(line >> (32 * c)) : 0u;
              const int from = row_lo - key0 - 32 * c;         // the group's first key that the row sees
              return from >= 32 ? 0u : info->there[c] & (from > 0 ? ~0u << from : ~0u);
            };
            auto value = [&](float s, const float2& f) {       // with the values' factor (NaN if it is)
              return fmaf(s, f.x * qs, fmaf(f.y, 0.f, static_cast<float>(static_cast<int>(__float_as_uint(f.y) >> 23) - 127)));
            };
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t seen = seen_of(c);
              tmem_ld32(ts + 32 * c, x);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((seen >> i) & 1u) most = fmaxf(most, value(x[i], info->key[32 * c + i]));
            }
            if (__any_sync(0xffffffffu, most + ref > kBSlack)) raise(most, j > w.j0);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t seen = seen_of(c);
              tmem_ld32(ts + 32 * c, x);
              tmem_ld_wait();
              uint32_t p[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float e[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float2 f = info->key[32 * c + 2 * i + h];
                  const bool in = (seen >> (2 * i + h)) & 1u;
                  e[h] = in ? ex2_approx(value(x[2 * i + h], f) + ref) : 0.f;
                  l = in ? fmaf(e[h], pow2_inverse(f.y) * kBSumUnit, l) : l;
                }
                const __half2 h2 = __floats2half2_rn(e[0], e[1]);
                p[i] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              tmem_st16(ts + 16 * c, p);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull + 8 * t);
        }
        // ---- the item's result, or this range's part of it
        wait_on(odone + 8 * t, (done - 1) & 1u, abort_flag, a.err);
        __syncwarp();
        tc_fence_after();
        const bool complete = w.j0 == 0 && w.j1 == w.seq.tiles;
        if (!there) l = 0.f;  // (whatever a row that is not there holds)
        const float g = l == 0.f ? 0.f : (complete ? kBSumUnit / l : 1.f);
        const int64_t slot = (static_cast<int64_t>(blockIdx.x) * 2 + (w.j0 > 0 ? 0 : 1)) * (2 * kWRows) + r;
        __nv_bfloat16* out = a.out + ((static_cast<int64_t>(w.b) * a.G + tok) * a.Hq + w.head * a.R + rr - tok * a.R) * D;
        float* part = a.part_o + slot * D;
        if (exists && !complete) a.part_ml[slot] = make_float2(ref != kBUnseen && there ? -ref : -INFINITY, l);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(to + c, o);
          tmem_ld_wait();
          if (!exists) continue;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = g != 0.f ? o[i] * g : 0.f;  // (O of a row that saw nothing is not looked at)
          if (complete) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // positions hold channels 0, 4, 1, 5, 2, 6, 3, 7 of a word
              uint32_t u[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int from = 8 * k + (i < 2 ? 4 * i : 4 * (i - 2) + 1);
                const __nv_bfloat162 v = __floats2bfloat162_rn(o[from], o[from + 2]);
                u[i] = *reinterpret_cast<const uint32_t*>(&v);
              }
              *reinterpret_cast<uint4*>(out + word_of_piece<D>(c / 8 + k) * 8) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              __stcg(reinterpret_cast<float4*>(part + c + i), make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
          }
        }
        tc_fence_before();
        if (threadIdx.x == 0 && w.j1 == w.seq.tiles) {
          const BlockParts parts(range.line, w.start, kWSetup, w.seq.tiles);
          wa.entry[(static_cast<int64_t>(w.b) * a.Hkv + w.head) * a.row_tiles + w.rt] = make_int2(parts.c0, parts.c1);
        }
      } else {
        it += static_cast<uint32_t>(w.j1 - w.j0);
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

// Joins the parts of items that several ranges share: a warp a row, 32 rows a CTA.
constexpr int kJoinRows = 32, kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv4_wide_join_kernel(const WideArgs wa) {
  const BlockArgs& a = wa.a;
  constexpr int kCtas = 2 * kWRows / kJoinRows, kE = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = static_cast<int>(blockIdx.x) / kCtas, rt = item % a.row_tiles, bh = item / a.row_tiles;
  const int b = bh / a.Hkv, head = bh - b * a.Hkv;
  pdl_trigger();
  pdl_wait();
  const int2 e = __ldg(wa.entry + item);
  if (e.x == e.y) return;  // (written by the range that had all of it)
  const int n = e.y - e.x + 1, nrows = min(a.tile_rows, a.rows - rt * a.tile_rows);
  for (int i = 0; i < kJoinRows / (kJoinThreads / 32); ++i) {
    const int r = (static_cast<int>(blockIdx.x) - item * kCtas) * kJoinRows + i * (kJoinThreads / 32) + warp;
    if (r >= nrows) break;
    auto slot = [&](int p) { return (static_cast<int64_t>(e.x + p) * 2 + (p == 0 ? 1 : 0)) * (2 * kWRows) + r; };
    float top = -INFINITY;
    for (int p = lane; p < n; p += 32) top = fmaxf(top, __ldcg(a.part_ml + slot(p)).x);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    float acc[kE] = {}, sum = 0.f;
    for (int p0 = 0; p0 < n; p0 += 32) {
      const float2 ml = p0 + lane < n ? __ldcg(a.part_ml + slot(p0 + lane)) : make_float2(-INFINITY, 0.f);
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
      sum = fmaf(f, ml.y, sum);
#pragma unroll 4
      for (int p = 0; p < min(32, n - p0); ++p) {
        const float weight = __shfl_sync(0xffffffffu, f, p);
        const float* from = a.part_o + slot(p0 + p) * D + lane * kE;
        float v[kE];
#pragma unroll
        for (int x = 0; x < kE; x += 2) {
          const float2 u = __ldcg(reinterpret_cast<const float2*>(from + x));
          v[x] = u.x;
          v[x + 1] = u.y;
        }
        if (weight != 0.f)  // (0: nothing of the row there)
#pragma unroll
          for (int x = 0; x < kE; ++x) acc[x] = fmaf(weight, v[x], acc[x]);
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
  p.total = p.entry + static_cast<size_t>(p.items) * sizeof(int2);
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
    e = launch_pdl(kv4_wide_join_kernel<D>, dim3(static_cast<unsigned>(p.items * (2 * kWRows / kJoinRows))), dim3(kJoinThreads), 0, st,
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
