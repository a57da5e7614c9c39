// The gated feed-forward sublayer (dflash2.ts #block: silu(gate(a)) * up(a), the MLP between a site's
// prepare and finish) and its gradients, on the tcgen05 tensor cores:
//
//   forward    g = x Wg^T, u = x Wu^T, h = act(g) * u                 x [M, H], Wg, Wu [F, H], h [M, F]
//   backward   dg = dh * u * act'(g), du = dh * act(g)                (one elementwise pass, bf16)
//              dx = dg Wg + du Wu;  dWg = dg^T x, dWu = du^T x
//
// with act(g) = g s(w(g)), s the logistic function and w(g) = g (silu) or 2 sqrt(2 / pi) (g + 0.044715 g^3)
// (gelu in its tanh form: (1 + tanh z) / 2 = s(2 z)).
//
// All three products run in one kernel on CTA pairs (cta_group::2) over 256 x 256 tiles:
//   forward: the pair's 256 weight rows are 128 rows of Wg (the leader's half) and the same 128 rows of
//            Wu (the peer's), so that a thread of the epilogue holds g and u of the same channels and
//            h leaves the kernel without g and u ever being stored (unless the caller keeps them).
//   dx:      K runs over the 2 F channels of (dg, du); the weights are read as they lie, [F, H], as an
//            operand whose H (not K) is contiguous ("MN-major").
//   dW:      K runs over the M rows; both operands are MN-major, so nothing is transposed in memory.
// Operands are 64-deep k-blocks in 128-byte-swizzled shared memory, filled by TMA through a ring of
// stages; the accumulator is double-buffered in TMEM (2 x 256 columns), so an epilogue overlaps the next
// tile's MMAs. Rows and columns past the matrices read as zeros and are not stored.
//
// Work: whole rounds of tiles go one tile per pair; what a last, partly filled round would leave idle is
// avoided by cutting the remaining tiles' k-blocks into equal shares, one per pair. A tile whose
// k-blocks fall to several pairs is finished by the pair that holds its last ones: the earlier pairs
// leave fp32 partial tiles in the workspace and raise flags, and the owner adds them in K order (so
// results do not depend on timing). Every pair takes its shares from the last piece to the first: the
// piece it gives away comes first, and an owner waits only for pairs of lower index, which were
// dispatched before it. The flags lie in the call's workspace and hold the call's own 64-bit number, so
// the workspace needs no initialisation and calls on different streams (with their own workspaces) are
// independent; an owner clears what it has read, so a captured call can be replayed.
//
// Bound: the tensor pipe, busy in 80 % of the cycles of a large product; the rest waits on operands from L2 (an
// SM takes 64 bytes a clock, a pair's tile needs 32 KB a CTA each 512 cycles). 1024 x 5120 x 13824 forward:
// 162 us, 1.80 PFLOP/s in a loop of 400 (a library product of the two weights at once: 151), 180 us among other
// passes; forward and all gradients of 4096 rows: 2.25 ms, 1.55 PFLOP/s under the power cap (library, sustained:
// 1.72).
#include <cuda_bf16.h>

#include <algorithm>

#include "ffn.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace dfl {
namespace {

constexpr int kFK = 64;                        // k per stage
constexpr int kFTile = 256;                    // rows and columns of a pair's tile
constexpr int kFHalf = 128 * 128;              // one CTA's half of an operand k-block, bytes
constexpr int kFStage = 2 * kFHalf;
constexpr int kFStages = 7;
constexpr int kFBar = 256;
constexpr int kFSmem = 1024 + kFStages * kFStage + kFBar;
constexpr int kFEpiWarps = 8;                  // two per 32 TMEM lanes, half of the columns each
constexpr int kFThreads = 64 + 32 * kFEpiWarps;  // warps: TMA, MMA, epilogue
constexpr int kFGroupM = 8;                    // tiles are walked in strips of 8 row tiles: neighbours share operands in L2
constexpr int kFSlot = 128 * kFTile;           // fp32 values of one CTA's partial tile
constexpr int kFMaxParts = 6;                  // pairs that share a tile at most, when there are few tiles
constexpr int kFMinPiece = 8;                  // k-blocks of a share at least
constexpr int kFMinGain = 45;                  // k-blocks a pair that shares of the last round have to save
constexpr int kFPitchBlocks = 32;              // k-blocks a pair from which x is copied to whole lines
constexpr uint64_t kFDrainNs = 100000000ull;

enum FfnMode { kForward = 0, kDx = 1, kDw = 2 };

struct FfnArgs {
  int M, H, F;
  int rows, cols;         // of the output: M x F (forward, per projection), M x H, F x H (per projection)
  int tiles_m, tiles_n, n_tiles;
  int kblocks;            // of one tile
  int kblocks0;           // dx: those of dg
  int a_rows;             // rows of a K-major A box: fewer than 128 when M is (the rest of the operand is not read out)
  int sk_tiles, sk_units; // tiles cut into shares, and the pairs that take them
  int act;
  __nv_bfloat16 *out0, *out1;  // h | dx | dWg, dWu
  uint32_t* pre;          // [M][F] kept g and u, or null
  float* slots;           // [CTA][64][128][4]: ffn_slot
  unsigned long long* flags;  // [CTA][epilogue warp]
  int wide;               // outputs take 32-byte stores (16-column rows, 32-byte aligned)
  unsigned long long call;
  int* err;
};
struct FfnMaps {
  CUtensorMap a0, a1, b0, b1;
};

// MN-major operand of 128-byte swizzled rows: 64 elements of M (or N) per row, one row per k, chunks
// of 64 columns `8192` bytes apart (64 k rows). Leading byte offset = the next 64 columns, stride
// byte offset = the next 8 k rows.
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8192 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}
__host__ __device__ constexpr uint32_t ffn_idesc(bool a_mn, bool b_mn) {
  return make_idesc(false, kFTile, kFTile) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}

// One piece of a pair's work: tile t, k-blocks [kb0, kb1).
struct FfnPiece {
  int t, kb0, kb1;
};
__device__ __forceinline__ long long ffn_share(const FfnArgs& a, int unit) {
  return static_cast<long long>(a.sk_tiles) * a.kblocks * unit / a.sk_units;
}
// Piece `idx` of pair `unit`: its share of the cut tiles from the last piece to the first, then whole tiles.
__device__ __forceinline__ bool ffn_piece(const FfnArgs& a, int unit, int units, int idx, FfnPiece& p) {
  int pieces = 0;
  if (unit < a.sk_units && a.sk_tiles > 0) {
    const long long s = ffn_share(a, unit), e = ffn_share(a, unit + 1);
    const int t0 = static_cast<int>(s / a.kblocks), t1 = static_cast<int>((e - 1) / a.kblocks);
    pieces = t1 - t0 + 1;
    if (idx < pieces) {
      p.t = t1 - idx;
      const long long first = static_cast<long long>(p.t) * a.kblocks;
      p.kb0 = static_cast<int>(max(s - first, 0LL));
      p.kb1 = static_cast<int>(min(e - first, static_cast<long long>(a.kblocks)));
      return true;
    }
  }
  const long long t = static_cast<long long>(a.sk_tiles) + unit + static_cast<long long>(idx - pieces) * units;
  if (t >= a.n_tiles) return false;
  p.t = static_cast<int>(t);
  p.kb0 = 0;
  p.kb1 = a.kblocks;
  return true;
}
// Tile -> (projection, row tile, column tile), walked in strips of kFGroupM row tiles.
__device__ __forceinline__ void ffn_tile(const FfnArgs& a, int t, int& proj, int& tm, int& tn) {
  const int per = a.tiles_m * a.tiles_n;
  proj = t / per;
  t -= proj * per;
  const int strip = t / (kFGroupM * a.tiles_n);
  const int left = min(kFGroupM, a.tiles_m - strip * kFGroupM);
  const int in = t - strip * kFGroupM * a.tiles_n;
  tn = in / left;
  tm = strip * kFGroupM + in - tn * left;
}

// Where row r's columns c .. c + 3 of a partial tile lie in its slot: [column / 4][row], so that a warp
// (32 rows, the same columns) moves 512 contiguous bytes.
__device__ __forceinline__ int ffn_slot(int r, int c) { return (c / 4 * 128 + r) * 4; }

__device__ __forceinline__ void ffn_abort(volatile int* abort_flag, int* err) {
  *abort_flag = 1;
  atomicCAS(err, 0, static_cast<int>(DFLASH2_ERR_TIMEOUT));
}
// Waits (bounded) until a partial tile's flag holds this call's number.
__device__ __forceinline__ bool ffn_wait_flag(const unsigned long long* flag, unsigned long long call,
                                              const volatile int* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1; ld_acquire_u64(flag) != call; ++i) {
    __nanosleep(64);
    if ((i & 15u) == 0u && (*abort_flag != 0 || globaltimer_ns() - t0 > kWaitLimitNs)) return false;
  }
  return true;
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// Stores 32 consecutive values of a row (columns col .. col + 31 of `cols`, a multiple of 8) as bf16.
__device__ __forceinline__ void ffn_store(__nv_bfloat16* row, int col, int cols, bool wide, const float (&y)[32]) {
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = ffn_pack(y[16 * v + 2 * j], y[16 * v + 2 * j + 1]);
    const int c = col + 16 * v;
    if (wide) {
      if (c < cols) st_global_v8(row + c, w);
    } else {
      if (c < cols) *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
      if (c + 8 < cols) *reinterpret_cast<uint4*>(row + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}
// The same for the kept products of 32 channels (32 words).
__device__ __forceinline__ void ffn_store_kept(uint32_t* row, int col, int cols, bool wide, const float (&g)[32],
                                               const float (&u)[32]) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = ffn_keep(g[8 * v + j], u[8 * v + j]);
    if (col + 8 * v >= cols) continue;
    if (wide) {
      st_global_v8(row + col + 8 * v, w);
    } else {
      *reinterpret_cast<uint4*>(row + col + 8 * v) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(row + col + 8 * v + 4) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

template <int kMode>
__global__ void __launch_bounds__(kFThreads, 1) ffn_kernel(const __grid_constant__ FfnMaps maps, const FfnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kFStages * kFStage);  // the leader's: both halves landed
  uint64_t* empty = full + kFStages;                                       // MMAs done reading the stage
  uint64_t* acc_full = empty + kFStages;                                   // [2]
  uint64_t* acc_empty = acc_full + 2;                                      // [2], the leader's
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int unit = static_cast<int>(blockIdx.x >> 1);
  const int units = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kFStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), 2 * kFEpiWarps);  // both CTAs' epilogue warps
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.a0);
    prefetch_tmap(&maps.b0);
    if (kMode != kForward) prefetch_tmap(&maps.a1);
    prefetch_tmap(&maps.b1);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers exist before the peer arrives on the leader's
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_trigger();
  pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      // L2: the operand that is read again stays, one that is read once goes first. A strip's rows are
      // done with when its columns fit about one round; the columns are read once if there is one strip
      // (1001 x 2568 x 6920: forward 91 -> 70 us, dx 100 -> 86, dW 122 -> 100; nothing at 4096 rows).
      const bool once = a.tiles_m <= kFGroupM;
      const uint64_t pol_a = kMode != kDw ? policy_evict_last()
                                          : (2 * kFGroupM * a.tiles_n <= 3 * units ? policy_evict_first() : policy_evict_normal());
      const uint64_t pol_b = kMode == kDw ? policy_evict_last() : (once ? policy_evict_first() : policy_evict_normal());
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      FfnPiece p;
      for (int idx = 0; ok && ffn_piece(a, unit, units, idx, p); ++idx) {
        int proj, tm, tn;
        ffn_tile(a, p.t, proj, tm, tn);
        // this CTA's 128 rows of A; its 128 columns of the output (B's rows)
        const int m0 = tm * kFTile + static_cast<int>(rank) * 128;
        const int n0 = kMode == kForward ? tn * 128 : tn * kFTile + static_cast<int>(rank) * 128;
        for (int kb = p.kb0; kb < p.kb1; ++kb) {
          if (!mbar_wait_bounded(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, kWaitLimitNs)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full[stage]);
          const uint32_t fbl = mapa_shared(fb, 0);  // both CTAs' copies complete on the leader's barrier
          if (rank == 0)
            mbar_arrive_expect_tx(fb, 2 * static_cast<uint32_t>(kMode == kDw ? kFStage : a.a_rows * 128 + kFHalf));
          const uint32_t sa = smem_u32(smem + stage * kFStage), sb = sa + kFHalf;
          if (kMode == kForward) {
            tma_load_2d_pair(sa, &maps.a0, fbl, kb * kFK, m0, pol_a);
            tma_load_2d_pair(sb, rank == 0 ? &maps.b0 : &maps.b1, fbl, kb * kFK, n0, pol_b);
          } else if (kMode == kDx) {
            const bool second = kb >= a.kblocks0;
            const int k = (second ? kb - a.kblocks0 : kb) * kFK;
            const CUtensorMap* mb = second ? &maps.b1 : &maps.b0;
            tma_load_2d_pair(sa, second ? &maps.a1 : &maps.a0, fbl, k, m0, pol_a);
            tma_load_2d_pair(sb, mb, fbl, n0, k, pol_b);
            tma_load_2d_pair(sb + kFHalf / 2, mb, fbl, n0 + 64, k, pol_b);
          } else {
            const CUtensorMap* ma = proj == 0 ? &maps.a0 : &maps.a1;
            tma_load_2d_pair(sa, ma, fbl, m0, kb * kFK, pol_a);
            tma_load_2d_pair(sa + kFHalf / 2, ma, fbl, m0 + 64, kb * kFK, pol_a);
            tma_load_2d_pair(sb, &maps.b0, fbl, n0, kb * kFK, pol_b);
            tma_load_2d_pair(sb + kFHalf / 2, &maps.b0, fbl, n0 + 64, kb * kFK, pol_b);
          }
          if (++stage == kFStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // copies in flight complete on the leader's barriers: give them a fixed time before leaving
        ffn_abort(abort_flag, a.err);
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (the leader's lane 0)
    if (lane == 0 && rank == 0) {
      constexpr bool kAMn = kMode == kDw, kBMn = kMode != kForward;
      constexpr uint32_t idesc = ffn_idesc(kAMn, kBMn);
      constexpr uint64_t kStepA = kAMn ? 16 * 128 / 16 : 2, kStepB = kBMn ? 16 * 128 / 16 : 2;  // 16 k further
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, any = false;
      FfnPiece p;
      for (int idx = 0; ok && ffn_piece(a, unit, units, idx, p); ++idx) {
        const int ab = idx & 1;
        if (!mbar_wait_bounded(smem_u32(&acc_empty[ab]), ((static_cast<uint32_t>(idx) >> 1) & 1u) ^ 1u, abort_flag,
                               kWaitLimitNs)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = p.kb0; kb < p.kb1; ++kb) {
          if (!mbar_wait_bounded(smem_u32(&full[stage]), phase, abort_flag, kWaitLimitNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * kFStage);
          const uint64_t adesc = kAMn ? desc_mnmajor_sw128(sa) : desc_kmajor_sw128(sa);
          const uint64_t bdesc = kBMn ? desc_mnmajor_sw128(sa + kFHalf) : desc_kmajor_sw128(sa + kFHalf);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_pair(tmem_base + static_cast<uint32_t>(ab * kFTile), adesc + kStepA * k, bdesc + kStepB * k, idesc,
                         (kb > p.kb0 || k > 0) ? 1u : 0u);
          mma_commit_pair(smem_u32(&empty[stage]), 0x3);  // frees the stage in both CTAs
          any = true;
          if (++stage == kFStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit_pair(smem_u32(&acc_full[ab]), 0x3);
      }
      if (!ok) {
        ffn_abort(abort_flag, a.err);
        if (any) {
          mma_commit_pair(smem_u32(drain), 0x1);
          mbar_wait_bounded(smem_u32(drain), 0, nullptr, kFDrainNs);
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;  // TMEM lanes 32 q ..
    const int ew = warp - 2, half = ew >> 2;  // its half of the columns
    const int cta = static_cast<int>(blockIdx.x);
    FfnPiece p;
    for (int idx = 0; ffn_piece(a, unit, units, idx, p); ++idx) {
      int proj, tm, tn;
      ffn_tile(a, p.t, proj, tm, tn);
      const int ab = idx & 1;
      const bool partial = p.kb1 < a.kblocks;
      // the pairs [u_first, unit) hold the tile's earlier k-blocks
      int u_first = unit;
      if (!partial && p.kb0 > 0) {
        const long long first = static_cast<long long>(p.t) * a.kblocks;
        while (u_first > 0 && ffn_share(a, u_first) > first) --u_first;
      }
      if (!mbar_wait_bounded_suspend(smem_u32(&acc_full[ab]), (static_cast<uint32_t>(idx) >> 1) & 1u, abort_flag,
                                     kWaitLimitNs)) {
        if (lane == 0) ffn_abort(abort_flag, a.err);
        break;
      }
      tc_fence_after();
      if (u_first < unit) {
        int got = 1;
        if (lane == 0)
          for (int u = u_first; got && u < unit; ++u)
            got = ffn_wait_flag(a.flags + (2 * u + static_cast<int>(rank)) * kFEpiWarps + ew, a.call, abort_flag) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          if (lane == 0) ffn_abort(abort_flag, a.err);
          break;
        }
      }
      const uint32_t tm0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(ab * kFTile);
      const int lrow = q * 32 + lane;                                // of the CTA's 128
      const int row = tm * kFTile + static_cast<int>(rank) * 128 + lrow;
      const bool valid = row < a.rows;
      // columns c0 .. c0 + 31 of the tile, the earlier pairs' parts included
      auto load = [&](int c0, float (&y)[32]) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32x32b_x32(tm0 + static_cast<uint32_t>(c0), r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(r[j]);
        if (u_first == unit || !valid) return;
        float sum[32] = {};
        for (int u = u_first; u < unit; ++u) {
          const float* src = a.slots + static_cast<size_t>(2 * u + static_cast<int>(rank)) * kFSlot;
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(src + ffn_slot(lrow, c0 + 4 * v)));
            sum[4 * v] += f.x; sum[4 * v + 1] += f.y; sum[4 * v + 2] += f.z; sum[4 * v + 3] += f.w;
          }
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] += sum[j];
      };
      if (partial) {
        // this warp's columns of the tile: for the forward pass half of g's and half of u's
        float* dst = a.slots + static_cast<size_t>(cta) * kFSlot;
        for (int i = 0; i < kFTile / 64; ++i) {
          const int c0 = kMode == kForward ? (i >> 1) * 128 + half * 64 + (i & 1) * 32 : half * 128 + i * 32;
          float y[32];
          load(c0, y);
          if (!valid) continue;
#pragma unroll
          for (int v = 0; v < 8; ++v)
            *reinterpret_cast<float4*>(dst + ffn_slot(lrow, c0 + 4 * v)) = make_float4(y[4 * v], y[4 * v + 1], y[4 * v + 2], y[4 * v + 3]);
        }
      } else if (kMode == kForward) {
        const size_t at = static_cast<size_t>(valid ? row : 0) * a.F;
        for (int c0 = half * 64; c0 < half * 64 + 64; c0 += 32) {
          float g[32], u[32];
          load(c0, g);
          load(128 + c0, u);
          const int col = tn * 128 + c0;
          if (valid && a.pre != nullptr) ffn_store_kept(a.pre + at, col, a.F, a.wide, g, u);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float slope;
            g[j] = g[j] * ffn_gate(g[j], a.act, slope) * u[j];
          }
          if (valid) ffn_store(a.out0 + at, col, a.F, a.wide, g);
        }
      } else {
        __nv_bfloat16* out = (proj == 0 ? a.out0 : a.out1) + static_cast<size_t>(valid ? row : 0) * a.cols;
        for (int c0 = half * 128; c0 < half * 128 + 128; c0 += 32) {
          float y[32];
          load(c0, y);
          if (valid) ffn_store(out, tn * kFTile + c0, a.cols, a.wide, y);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[ab]), 0));
      if (partial) {
        __threadfence();  // every lane's rows are visible before the flag
        __syncwarp();
        if (lane == 0) st_release_u64(a.flags + cta * kFEpiWarps + ew, a.call);
      }
      if (lane == 0)  // read: ready for a replay
        for (int u = u_first; u < unit; ++u) a.flags[(2 * u + static_cast<int>(rank)) * kFEpiWarps + ew] = 0ull;
    }
  }

  tc_fence_before();
  cluster_sync_all();  // no MMA, commit or remote arrival is in flight towards either CTA
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// Row of element i of rows of n (a 64-bit division is some hundred instructions).
__device__ __forceinline__ size_t ffn_row(size_t i, uint32_t n) {
  return i <= 0xffffffffu ? static_cast<uint32_t>(i) / n : i / n;
}

// dg = dh u act'(g), du = dh act(g), rounded to bf16 (the operands of the products): thread = 8
// channels of one row; out [2][M][ffn_pitch(F)].
__global__ void __launch_bounds__(256)
    ffn_gate_grad_kernel(const __nv_bfloat16* __restrict__ dh, const uint32_t* __restrict__ pre, size_t n8, int act,
                         uint32_t cols8, uint32_t pitch8, size_t plane8, __nv_bfloat16* __restrict__ dgu) {
  pdl_trigger();
  pdl_wait();
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n8) return;
  const uint4 d4 = __ldg(reinterpret_cast<const uint4*>(dh) + i);
  const uint4 p4[2] = {__ldg(reinterpret_cast<const uint4*>(pre) + 2 * i),
                       __ldg(reinterpret_cast<const uint4*>(pre) + 2 * i + 1)};
  const uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w};
  const uint32_t pw[8] = {p4[0].x, p4[0].y, p4[0].z, p4[0].w, p4[1].x, p4[1].y, p4[1].z, p4[1].w};
  uint32_t og[4], ou[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 d = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&dw[j]));
    const float dd[2] = {d.x, d.y};
    float dg[2], du[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t w = pw[2 * j + e];
      const float g = ffn_kept1(w & 0xffffu), u = ffn_kept1(w >> 16);
      float slope;
      const float s = ffn_gate(g, act, slope);
      dg[e] = dd[e] * u * fmaf(g * s * (1.f - s), slope, s);
      du[e] = dd[e] * g * s;
    }
    og[j] = ffn_pack(dg[0], dg[1]);
    ou[j] = ffn_pack(du[0], du[1]);
  }
  const size_t at = i + ffn_row(i, cols8) * (pitch8 - cols8);
  reinterpret_cast<uint4*>(dgu)[at] = make_uint4(og[0], og[1], og[2], og[3]);
  reinterpret_cast<uint4*>(dgu)[plane8 + at] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
}

// Rows of a pitch that the copy engine likes (see ffn_pitch).
__global__ void __launch_bounds__(256)
    ffn_pitch_kernel(const __nv_bfloat16* __restrict__ x, size_t n8, uint32_t cols8, uint32_t pitch8,
                     __nv_bfloat16* __restrict__ y) {
  pdl_trigger();
  pdl_wait();
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n8) reinterpret_cast<uint4*>(y)[i + ffn_row(i, cols8) * (pitch8 - cols8)] = __ldg(reinterpret_cast<const uint4*>(x) + i);
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
int ffn_units(int sms) { return std::max(1, sms / 2); }

size_t ffn_share_bytes(int sms) {
  const size_t ctas = 2 * static_cast<size_t>(ffn_units(sms));
  return align256(ctas * kFSlot * sizeof(float)) + align256(ctas * kFEpiWarps * sizeof(unsigned long long));
}

template <int kMode>
int launch_ffn_gemm(const FfnMaps& maps, FfnArgs a, void* share_ws, cudaStream_t st) {
  const int units = ffn_units(sm_count());
  a.slots = static_cast<float*>(share_ws);
  a.flags = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(share_ws) +
                                                  align256(2 * static_cast<size_t>(units) * kFSlot * sizeof(float)));
  a.call = next_call_number();
  auto is32 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; };
  a.wide = a.cols % 16 == 0 && is32(a.out0) && is32(a.out1) && is32(a.pre);
  a.err = device_error_word();
  if (a.err == nullptr) return fail(DFLASH2_ERR_CUDA, "no device error word");
  // The last round's tiles are cut into shares where that saves each pair kFMinGain k-blocks (a cut tile costs
  // its partial sums' way through the workspace: with 5 saved, 333 x 1352 x 3592 takes 25.0 us cut and 14.8
  // whole; with 25, 1024 x 5120 x 13824 takes 195 and 183; a third size, 1001 x 2568 x 6920, agrees). Few
  // tiles over all pairs would leave an owner many parts to add (19 of them at 1024 x 5120 with K = 27648:
  // 320 us against 142 us of MMAs), so the round before is cut with them where there is one: then a share is a
  // tile and a bit, and a tile has at most three parts. Without one, at most kFMaxParts pairs share a tile. A
  // share has at least kFMinPiece k-blocks.
  const int rest = a.n_tiles % units;
  a.sk_tiles = static_cast<long long>(a.kblocks) * (units - rest) < kFMinGain * units ? 0 : rest;
  if (a.sk_tiles > 0 && 3 * rest < units && a.n_tiles > units) a.sk_tiles += units;
  const long long total = static_cast<long long>(a.sk_tiles) * a.kblocks;
  a.sk_units = static_cast<int>(std::max<long long>(
      1, std::min({static_cast<long long>(units), total / kFMinPiece, static_cast<long long>(a.sk_tiles) * kFMaxParts})));
  if (a.sk_units < units && a.sk_units <= a.sk_tiles) a.sk_tiles = 0;  // K too short to cut
  const int grid = 2 * std::min(units, a.sk_tiles > 0 ? std::max(a.sk_units, a.n_tiles - a.sk_tiles) : a.n_tiles);
  static unsigned done = 0;
  auto kern = ffn_kernel<kMode>;
  if (!ensure_smem_attr(kern, kFSmem, &done)) return fail(DFLASH2_ERR_CUDA, "cudaFuncSetAttribute failed (gated FFN)");
  cudaLaunchAttribute cl[1];
  cl[0].id = cudaLaunchAttributeClusterDimension;
  cl[0].val.clusterDim.x = 2;
  cl[0].val.clusterDim.y = 1;
  cl[0].val.clusterDim.z = 1;
  const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kFThreads), kFSmem, st, cl, 1, maps, a);
  return e == cudaSuccess ? DFLASH2_OK : fail(DFLASH2_ERR_CUDA, "gated FFN launch failed: %s", cudaGetErrorString(e));
}

int tiles_of(int n, int tile) { return static_cast<int>((static_cast<long long>(n) + tile - 1) / tile); }

bool ffn_map(CUtensorMap* m, const void* p, int rows, int cols, int box_rows, int pitch = 0) {
  return make_tmap_sw128(m, p, static_cast<uint64_t>(rows), static_cast<uint64_t>(cols), static_cast<uint32_t>(box_rows),
                         static_cast<uint64_t>(pitch));
}

// Elements between the rows of an operand that lies in the workspace: whole lines of 128 bytes. Where they are
// not, each of a box's rows crosses two lines, and L2, whose 64 bytes a clock an SM needs in full, is asked
// twice. x is copied to such rows where its own are not; the weights are read as they lie (a copy of them
// costs what it gives at a thousand rows).
// 1001 x 2568 x 6920, forward and gradients: 247 -> 213 us. A forward product of less than kFPitchBlocks k-blocks a
// pair keeps x as it is: 333 x 1352 x 3592 (17 of them) is 1.2 us slower with the copy.
int ffn_pitch(int n) { return (n + 63) / 64 * 64; }
size_t ffn_pitch_bytes(int M, int n) { return n % 64 == 0 ? 0 : align256(static_cast<size_t>(M) * ffn_pitch(n) * 2); }

cudaError_t launch_ffn_pitch(const void* x, int M, int n, void* y, cudaStream_t st) {
  const size_t n8 = static_cast<size_t>(M) * n / 8;
  return launch_pdl(ffn_pitch_kernel, dim3(static_cast<unsigned>((n8 + 255) / 256)), dim3(256), 0, st, nullptr, 0,
                    static_cast<const __nv_bfloat16*>(x), n8, static_cast<uint32_t>(n / 8),
                    static_cast<uint32_t>(ffn_pitch(n) / 8), static_cast<__nv_bfloat16*>(y));
}

}  // namespace

// Workspace: [partial tiles][flags][x in whole lines, if its rows are not] and, for the backward pass, [dg, du].
size_t gated_ffn_workspace(int M, int H, int F, bool backward, int sms) {
  return ffn_share_bytes(sms) + ffn_pitch_bytes(M, H) + (backward ? align256(2 * static_cast<size_t>(M) * ffn_pitch(F) * 2) : 0);
}

int launch_gated_ffn(const GatedFfn& r, cudaStream_t st) {
  if (r.M <= kFfnSmallRows) return launch_gated_ffn_small(r, st);
  FfnMaps maps;
  const int a_rows = (std::min(128, r.M) + 7) / 8 * 8;
  const void* x = r.x;
  int pitch = r.H;
  const long long blocks = static_cast<long long>(tiles_of(r.M, kFTile)) * tiles_of(r.F, 128) * tiles_of(r.H, kFK);
  if (r.H % 64 != 0 && blocks > static_cast<long long>(kFPitchBlocks) * ffn_units(sm_count())) {
    void* y = static_cast<uint8_t*>(r.workspace) + ffn_share_bytes(sm_count());
    const cudaError_t e = launch_ffn_pitch(x, r.M, r.H, y, st);
    if (e != cudaSuccess) return fail(DFLASH2_ERR_CUDA, "gated FFN row copy failed: %s", cudaGetErrorString(e));
    x = y;
    pitch = ffn_pitch(r.H);
  }
  if (!ffn_map(&maps.a0, x, r.M, r.H, a_rows, pitch) || !ffn_map(&maps.b0, r.w_gate, r.F, r.H, 128) ||
      !ffn_map(&maps.b1, r.w_up, r.F, r.H, 128))
    return fail(DFLASH2_ERR_CUDA, "tensor map encode failed (gated FFN)");
  maps.a1 = maps.a0;
  FfnArgs a{};
  a.M = r.M; a.H = r.H; a.F = r.F;
  a.rows = r.M;
  a.cols = r.F;
  a.a_rows = a_rows;
  a.tiles_m = tiles_of(r.M, kFTile);
  a.tiles_n = tiles_of(r.F, 128);
  a.n_tiles = a.tiles_m * a.tiles_n;
  a.kblocks = tiles_of(r.H, kFK);
  a.act = r.act;
  a.out0 = static_cast<__nv_bfloat16*>(r.h);
  a.pre = static_cast<uint32_t*>(r.pre);
  return launch_ffn_gemm<kForward>(maps, a, r.workspace, st);
}

int launch_gated_ffn_backward(const GatedFfn& r, cudaStream_t st) {
  uint8_t* rows = static_cast<uint8_t*>(r.workspace) + ffn_share_bytes(sm_count());  // x's, then dg's and du's
  __nv_bfloat16* dgu = reinterpret_cast<__nv_bfloat16*>(rows + ffn_pitch_bytes(r.M, r.H));
  const int pitch = ffn_pitch(r.F);
  const size_t plane = static_cast<size_t>(r.M) * pitch;
  const size_t n8 = static_cast<size_t>(r.M) * r.F / 8;
  const cudaError_t e =
      launch_pdl(ffn_gate_grad_kernel, dim3(static_cast<unsigned>((n8 + 255) / 256)), dim3(256), 0, st, nullptr, 0,
                 static_cast<const __nv_bfloat16*>(r.dh), static_cast<const uint32_t*>(r.pre), n8, r.act,
                 static_cast<uint32_t>(r.F / 8), static_cast<uint32_t>(pitch / 8), plane / 8, dgu);
  if (e != cudaSuccess) return fail(DFLASH2_ERR_CUDA, "gated FFN gradient launch failed: %s", cudaGetErrorString(e));
  FfnArgs a{};
  a.M = r.M; a.H = r.H; a.F = r.F;
  a.cols = r.H;
  a.tiles_n = tiles_of(r.H, kFTile);
  FfnMaps maps;
  if (r.dx != nullptr) {
    a.a_rows = (std::min(128, r.M) + 7) / 8 * 8;
    if (!ffn_map(&maps.a0, dgu, r.M, r.F, a.a_rows, pitch) || !ffn_map(&maps.a1, dgu + plane, r.M, r.F, a.a_rows, pitch) ||
        !ffn_map(&maps.b0, r.w_gate, r.F, r.H, kFK) || !ffn_map(&maps.b1, r.w_up, r.F, r.H, kFK))
      return fail(DFLASH2_ERR_CUDA, "tensor map encode failed (gated FFN dx)");
    a.rows = r.M;
    a.tiles_m = tiles_of(r.M, kFTile);
    a.n_tiles = a.tiles_m * a.tiles_n;
    a.kblocks0 = tiles_of(r.F, kFK);
    a.kblocks = 2 * a.kblocks0;
    a.out0 = a.out1 = static_cast<__nv_bfloat16*>(r.dx);
    const int rc = launch_ffn_gemm<kDx>(maps, a, r.workspace, st);
    if (rc != DFLASH2_OK) return rc;
  }
  if (r.dw_gate != nullptr) {
    const void* x = r.x;
    if (r.H % 64 != 0) {
      const cudaError_t e1 = launch_ffn_pitch(x, r.M, r.H, rows, st);
      if (e1 != cudaSuccess) return fail(DFLASH2_ERR_CUDA, "gated FFN row copy failed: %s", cudaGetErrorString(e1));
      x = rows;
    }
    if (!ffn_map(&maps.a0, dgu, r.M, r.F, kFK, pitch) || !ffn_map(&maps.a1, dgu + plane, r.M, r.F, kFK, pitch) ||
        !ffn_map(&maps.b0, x, r.M, r.H, kFK, ffn_pitch(r.H)))
      return fail(DFLASH2_ERR_CUDA, "tensor map encode failed (gated FFN dW)");
    maps.b1 = maps.b0;
    a.rows = r.F;
    a.tiles_m = tiles_of(r.F, kFTile);
    a.n_tiles = 2 * a.tiles_m * a.tiles_n;
    a.kblocks = tiles_of(r.M, kFK);
    a.out0 = static_cast<__nv_bfloat16*>(r.dw_gate);
    a.out1 = static_cast<__nv_bfloat16*>(r.dw_up);
    return launch_ffn_gemm<kDw>(maps, a, r.workspace, st);
  }
  return DFLASH2_OK;
}

}  // namespace dfl
