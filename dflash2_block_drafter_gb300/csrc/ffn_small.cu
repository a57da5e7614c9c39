// The gated feed-forward product h = act(x Wg^T) * (x Wu^T) for up to 128 rows (one token to eight draft
// blocks): a stream of the two weights. The operands are swapped, so that the weights fill the
// tensor core's 128-row side whatever the number of rows: a CTA's tile is 64 rows of Wg and the same
// 64 rows of Wu over the np <= 128 (padded to 16) rows of x, accumulated in TMEM over k-blocks of 64
// that a ring of TMA stages brings. The tile then crosses shared memory, where a thread picks up g
// and u of eight channels of one row and stores h.
//
// All tiles are resident at once (two or three CTAs an SM), so that every SM keeps copies in flight until
// the stream ends. Few tiles (a small F) split K over the CTAs of a cluster; the parts are read through
// distributed shared memory and added in K order.
//
// Bound: the weights' stream. 16 rows, 2 x 13824 x 5120 weights (283 MB): 44 us, 6.4 TB/s.
#include <cuda_bf16.h>

#include <algorithm>

#include "ffn.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace dfl {
namespace {

constexpr int kSK = 64;                    // k per stage
constexpr int kSRows = 64;                 // channels of a tile
constexpr int kSWBytes = 2 * kSRows * 128; // weight bytes of a stage
constexpr int kSThreads = 192;             // warps: TMA, MMA, 4 x epilogue
constexpr int kSBar = 256;
constexpr int kSMaxStages = 8;
constexpr uint64_t kSDrainNs = 100000000ull;

struct SmallArgs {
  int M, F, np, kblocks, ks, stages, act;
  int body;  // bytes of the stages, or of the tile that replaces them
  uint32_t tmem_cols;
  __nv_bfloat16* h;
  uint32_t* pre;
  int* err;
};
struct SmallMaps {
  CUtensorMap x, wg, wu;
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kSThreads) ffn_small_kernel(const __grid_constant__ SmallMaps maps, const SmallArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int stage_bytes = kSWBytes + a.np * 128;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + a.body);
  uint64_t* empty = full + kSMaxStages;
  uint64_t* acc_full = empty + kSMaxStages;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = a.ks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int f0 = (static_cast<int>(blockIdx.x) / a.ks) * kSRows;
  const int kb0 = a.kblocks * rank / a.ks, kb1 = a.kblocks * (rank + 1) / a.ks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(acc_full), 1);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.x);
    prefetch_tmap(&maps.wg);
    prefetch_tmap(&maps.wu);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), a.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_trigger();
  pdl_wait();

  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_w = policy_evict_first();  // read once
      const uint64_t pol_x = policy_evict_last();   // read by every CTA
      const uint32_t bytes = static_cast<uint32_t>(stage_bytes);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_bounded(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, kWaitLimitNs)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(&full[stage]);
        const uint32_t sw = smem_u32(smem + stage * stage_bytes);
        mbar_arrive_expect_tx(fb, bytes);
        tma_load_2d(sw, &maps.wg, fb, kb * kSK, f0, pol_w);
        tma_load_2d(sw + kSWBytes / 2, &maps.wu, fb, kb * kSK, f0, pol_w);
        tma_load_2d(sw + kSWBytes, &maps.x, fb, kb * kSK, 0, pol_x);
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {  // copies in flight land before the CTA leaves
        *abort_flag = 1;
        atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_TIMEOUT));
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc(false, 128, a.np);
      int stage = 0;
      uint32_t phase = 0;
      bool any = false;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_bounded(smem_u32(&full[stage]), phase, abort_flag, kWaitLimitNs)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sw = smem_u32(smem + stage * stage_bytes);
        const uint64_t adesc = desc_kmajor_sw128(sw), bdesc = desc_kmajor_sw128(sw + kSWBytes);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16(tmem_base, adesc + 2 * k, bdesc + 2 * k, idesc, (kb > kb0 || k > 0) ? 1u : 0u);
        mma_commit(smem_u32(&empty[stage]));
        any = true;
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) {
        mma_commit(smem_u32(acc_full));
      } else {
        *abort_flag = 1;
        atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_TIMEOUT));
        if (any) {
          mma_commit(smem_u32(drain));
          mbar_wait_bounded(smem_u32(drain), 0, nullptr, kSDrainNs);
        }
      }
    }
    __syncwarp();
  }
  // The tile through shared memory (the stages are read out once the accumulator is complete):
  // P[weight row][x row], an odd pitch so that neighbouring weight rows fall into different banks.
  float* P = reinterpret_cast<float*>(smem);
  const int pitch = a.np + 1;
  bool good = true;
  if (warp >= 2) {
    const int q = warp & 3;
    good = mbar_wait_bounded_suspend(smem_u32(acc_full), 0, abort_flag, kWaitLimitNs);
    if (!good && lane == 0) {
      *abort_flag = 1;
      atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_TIMEOUT));
    }
    if (good) {
      tc_fence_after();
      for (int c0 = 0; c0 < a.np; c0 += 16) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c0), r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) P[(q * 32 + lane) * pitch + c0 + j] = __uint_as_float(r[j]);
      }
    }
  }
  if (a.ks > 1)
    cluster_sync_all();
  else
    __syncthreads();
  if (*abort_flag == 0) {
    const uint32_t p0 = smem_u32(P);
    for (int i = rank * kSThreads + threadIdx.x; i < a.M * (kSRows / 8); i += a.ks * kSThreads) {
      const int m = i / (kSRows / 8), c = (i % (kSRows / 8)) * 8;
      if (f0 + c >= a.F) continue;
      float g[8], u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] = P[(c + j) * pitch + m];
        u[j] = P[(kSRows + c + j) * pitch + m];
      }
      if (a.ks > 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          g[j] = u[j] = 0.f;
          for (int s = 0; s < a.ks; ++s) {
            const uint32_t at = mapa_shared(p0, static_cast<uint32_t>(s));
            g[j] += ld_cluster_f32(at + static_cast<uint32_t>((c + j) * pitch + m) * 4);
            u[j] += ld_cluster_f32(at + static_cast<uint32_t>((kSRows + c + j) * pitch + m) * 4);
          }
        }
      }
      const size_t at = static_cast<size_t>(m) * a.F + f0 + c;
      if (a.pre != nullptr) {
#pragma unroll
        for (int v = 0; v < 2; ++v)
          *reinterpret_cast<uint4*>(a.pre + at + 4 * v) =
              make_uint4(ffn_keep(g[4 * v], u[4 * v]), ffn_keep(g[4 * v + 1], u[4 * v + 1]),
                         ffn_keep(g[4 * v + 2], u[4 * v + 2]), ffn_keep(g[4 * v + 3], u[4 * v + 3]));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float slope;
        g[j] = g[j] * ffn_gate(g[j], a.act, slope) * u[j];
      }
      *reinterpret_cast<uint4*>(a.h + at) =
          make_uint4(ffn_pack(g[0], g[1]), ffn_pack(g[2], g[3]), ffn_pack(g[4], g[5]), ffn_pack(g[6], g[7]));
    }
  }
  tc_fence_before();
  if (a.ks > 1)
    cluster_sync_all();  // no CTA leaves while a peer reads its part
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, a.tmem_cols);
  }
}

}  // namespace

int launch_gated_ffn_small(const GatedFfn& r, cudaStream_t st) {
  SmallArgs a{};
  a.M = r.M;
  a.F = r.F;
  a.np = (r.M + 15) / 16 * 16;
  a.kblocks = (r.H + kSK - 1) / kSK;
  a.act = r.act;
  a.tmem_cols = a.np <= 32 ? 32u : (a.np <= 64 ? 64u : 128u);
  a.h = static_cast<__nv_bfloat16*>(r.h);
  a.pre = static_cast<uint32_t*>(r.pre);
  a.err = device_error_word();
  if (a.err == nullptr) return fail(DFLASH2_ERR_CUDA, "no device error word");
  SmallMaps maps;
  if (!make_tmap_sw128(&maps.x, r.x, static_cast<uint64_t>(r.M), static_cast<uint64_t>(r.H), static_cast<uint32_t>(a.np)) ||
      !make_tmap_sw128(&maps.wg, r.w_gate, static_cast<uint64_t>(r.F), static_cast<uint64_t>(r.H), kSRows) ||
      !make_tmap_sw128(&maps.wu, r.w_up, static_cast<uint64_t>(r.F), static_cast<uint64_t>(r.H), kSRows))
    return fail(DFLASH2_ERR_CUDA, "tensor map encode failed (gated FFN)");
  const int sms = sm_count();
  const int tiles = (r.F + kSRows - 1) / kSRows;
  // K splits: two CTAs an SM at most, at least four k-blocks each
  a.ks = std::max(1, std::min({8, 2 * sms / tiles, a.kblocks / 4}));
  const int ctas = tiles * a.ks;
  const int stage_bytes = kSWBytes + a.np * 128;
  // two CTAs an SM share its shared memory (three when that many are needed to have every tile resident)
  const int per_sm = ctas <= sms ? 1 : (ctas <= 2 * sms ? 2 : 3);
  const int room = 232448 / per_sm - 1024 - 1024 - kSBar;
  a.stages = std::max(2, std::min(kSMaxStages, room / stage_bytes));
  a.body = std::max(a.stages * stage_bytes, 128 * (a.np + 1) * 4);
  const int smem = 1024 + a.body + kSBar;
  static unsigned done = 0;
  if (!ensure_smem_attr(ffn_small_kernel, 232448, &done))
    return fail(DFLASH2_ERR_CUDA, "cudaFuncSetAttribute failed (gated FFN)");
  cudaLaunchAttribute cl[1];
  cl[0].id = cudaLaunchAttributeClusterDimension;
  cl[0].val.clusterDim.x = static_cast<unsigned>(a.ks);
  cl[0].val.clusterDim.y = 1;
  cl[0].val.clusterDim.z = 1;
  const cudaError_t e = launch_pdl(ffn_small_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kSThreads),
                                   static_cast<size_t>(smem), st, cl, 1, maps, a);
  return e == cudaSuccess ? DFLASH2_OK : fail(DFLASH2_ERR_CUDA, "gated FFN launch failed: %s", cudaGetErrorString(e));
}

}  // namespace dfl
