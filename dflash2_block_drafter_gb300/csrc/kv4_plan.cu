// Pages and slots of a paged cache, planned on the GPU: what each sequence gains or drops becomes page-table
// entries, slots of new rows and a queue of free pages.
//
// Sequence b holds L tokens in ceil(L / p) pages and changes by c: it needs max(0, ceil((L + c) / p) - ceil(L / p))
// pages more, or gives as many back. Where its pages and rows lie among all is a prefix sum over the sequences; every
// page and every row then finds its sequence by a binary search of those sums and writes its own entry.
//
// A sequence is granted if its pages fit the queue, and its rows the output, together with those of all sequences
// before it. The sums run over refused sequences too, so that what is granted is a prefix of those that ask, and
// each sum cut off at the largest granted one gives the granted sequences' places.
//
// What bounds it: latency. 64 sequences' blocks of 16 rows take 5.3 us in a graph, a launch and four passes over
// shared memory; 98304 packed rows 12 us and 4096 sequences 11.3, of which the cluster's start and end and the three
// scans are most (the rows' bytes, 1.2 MB, would take 0.2).
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace dfl {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;  // CTAs, of a call with many sequences or rows

struct PlanArgs {
  const int32_t *ctx, *change, *state, *place;
  int32_t *table, *queue, *ctx_out, *state_out, *offsets, *positions;
  int64_t* slots;
  int B, width, page_shift, num_pages, capacity, G, rows;
  int* err;
};

struct PlanSums {
  long long taken, given, rows;
};

// Exclusive sums over the block's threads, and the total (all threads call it).
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = x;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, m);
    if (lane >= m) inc += v;
  }
  __syncthreads();  // (the sums of a scan before have been read)
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  long long mine = warp_sums[lane];
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, mine, m);
    if (lane >= m) mine += v;
  }
  total = __shfl_sync(0xffffffffu, mine, 31);
  const long long before = __shfl_sync(0xffffffffu, mine, max(0, warp - 1));
  return (warp > 0 ? before : 0) + inc - x;
}

// The first b with end[b] > i (end ascends; i is below the last).
__device__ __forceinline__ int owner_of(const int* end, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > i)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(const PlanArgs a) {
  extern __shared__ int plan_smem[];
  int* ctx = plan_smem;          // [B] lengths before
  int* taken = ctx + a.B;        // [B] sums over the sequences up to this one: pages taken,
  int* given = taken + a.B;      // pages given back,
  int* row_end = given + a.B;    // rows
  __shared__ long long warp_sums[32];
  __shared__ int most[3];        // the largest granted sums
  const int tid = static_cast<int>(threadIdx.x);
  const int me = static_cast<int>(blockIdx.x) * kPlanThreads + tid, all = static_cast<int>(gridDim.x) * kPlanThreads;
  const bool leads = blockIdx.x == 0;
  pdl_trigger();
  pdl_wait();
  const int page = 1 << a.page_shift;
  const long long cap = static_cast<long long>(a.width) << a.page_shift;
  // (ordinary loads, not the read-only path's: lengths and state may be outputs too)
  int head = a.state[0], count = a.state[1];
  const bool state_ok = head >= 0 && head < a.capacity && count >= 0 && count <= a.capacity;
  if (!state_ok && tid == 0) atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_INVALID_ARG));
  if (tid < 3) most[tid] = 0;

  auto pages_of = [&](int n) { return static_cast<int>((static_cast<unsigned>(n) + page - 1) >> a.page_shift); };
  // what each sequence asks for: pages (more, or fewer) and tokens; nothing fits a length outside its pages
  constexpr int kBad = -0x7fffffff - 1;
  for (int b = tid; b < a.B; b += kPlanThreads) {
    const int len = a.ctx[b], change = a.change[b];
    const long long end = static_cast<long long>(len) + change;
    const bool fits = state_ok && len >= 0 && len <= cap && end >= 0 && end <= cap;
    if (!fits) atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_INVALID_ARG));
    ctx[b] = len;
    taken[b] = fits ? pages_of(static_cast<int>(end)) - pages_of(len) : kBad;
    row_end[b] = fits ? change : 0;
  }
  __syncthreads();
  // sums: each thread a run of sequences
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long need = 0, back = 0;
  for (int b = b0; b < b1; ++b) {
    const int d = taken[b];
    need += max(0, d);
    back += d == kBad ? 0 : max(0, -d);
  }
  long long total;
  const long long need0 = block_scan(need, warp_sums, total), back0 = block_scan(back, warp_sums, total);
  // the pages decide first: a sequence that gets none asks for no rows
  auto granted_pages = [&](int d, long long need_sum, long long back_sum) {
    if (d > 0) return need_sum <= count;
    if (d < 0) return d != kBad && back_sum <= a.capacity - count;
    return true;
  };
  long long rows = 0;
  need = need0;
  back = back0;
  for (int b = b0; b < b1; ++b) {
    const int d = taken[b];
    need += max(0, d);
    back += d == kBad ? 0 : max(0, -d);
    if (granted_pages(d, need, back))
      rows += max(0, row_end[b]);
    else if (d < 0)  // more pages come back than there can be
      atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_INVALID_ARG));
  }
  rows = block_scan(rows, warp_sums, total);
  // then the rows
  need = need0;
  back = back0;
  int last[3] = {0, 0, 0};  // the thread's largest granted sums
  for (int b = b0; b < b1; ++b) {
    const int d = taken[b], gain = row_end[b];
    need += max(0, d);
    back += d == kBad ? 0 : max(0, -d);
    bool granted = granted_pages(d, need, back);
    if (granted && gain > 0) {
      rows += gain;
      granted = rows <= a.rows;
    }
    if (granted && d > 0) last[0] = static_cast<int>(need);
    if (granted && d < 0) last[1] = static_cast<int>(back);
    if (granted && gain > 0) last[2] = static_cast<int>(rows);
    taken[b] = static_cast<int>(min(need, 0x7fffffffll));
    given[b] = static_cast<int>(min(back, 0x7fffffffll));
    row_end[b] = static_cast<int>(min(rows, 0x7fffffffll));
  }
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    last[x] = __reduce_max_sync(0xffffffffu, last[x]);
    if ((tid & 31) == 0) atomicMax(most + x, last[x]);
  }
  __syncthreads();
  const int pages_taken = most[0], pages_given = most[1], rows_all = most[2];
  for (int b = tid; b < a.B; b += kPlanThreads) {
    taken[b] = min(taken[b], pages_taken);
    given[b] = min(given[b], pages_given);
    row_end[b] = min(row_end[b], rows_all);
  }
  __syncthreads();
  auto before = [](const int* end, int b) { return b > 0 ? end[b - 1] : 0; };
  // entry i of the pages waiting (i < 2 capacity)
  auto place_in_queue = [&](int i) {
    const long long at = static_cast<long long>(head) + i;
    return static_cast<int>(at >= a.capacity ? at - a.capacity : at);
  };
  auto page_ok = [&](int p) {
    if (p >= 0 && p < a.num_pages) return true;
    atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_BAD_INDEX));
    return false;
  };
  for (int i = me; i < pages_taken; i += all) {
    const int b = owner_of(taken, a.B, i);
    const int p = a.queue[place_in_queue(i)];
    page_ok(p);
    a.table[static_cast<long long>(b) * a.width + pages_of(ctx[b]) + (i - before(taken, b))] = p;
  }
  for (int i = me; i < pages_given; i += all) {
    const int b = owner_of(given, a.B, i);
    const int n = given[b] - before(given, b);  // the sequence's last pages
    const int p = a.table[static_cast<long long>(b) * a.width + pages_of(ctx[b]) - n + (i - before(given, b))];
    page_ok(p);
    a.queue[place_in_queue(count + i)] = p;
  }
  const int items = a.place != nullptr ? a.B * a.G : a.rows;
  for (int i = me; i < items; i += all) {
    int b = 0, j = -1;
    bool there;
    if (a.place != nullptr) {
      b = i / a.G;
      j = a.place[i];
      there = j >= 0 && j < row_end[b] - before(row_end, b);
    } else {
      there = i < rows_all;
      if (there) {
        b = owner_of(row_end, a.B, i);
        j = i - before(row_end, b);
      }
    }
    int64_t slot = -1;
    int pos = -1;
    if (there) {
      pos = ctx[b] + j;
      const int k = pos >> a.page_shift, have = static_cast<int>(pages_of(ctx[b]));
      const int p = k < have ? a.table[static_cast<long long>(b) * a.width + k]
                             : a.queue[place_in_queue(before(taken, b) + (k - have))];
      if (page_ok(p)) slot = (static_cast<int64_t>(p) << a.page_shift) + (pos & (page - 1));
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
  if (gridDim.x > 1) cluster_sync_all();  // (the outputs may be the inputs' own buffers: every CTA has read them)
  for (int b = me; b < a.B; b += all) {
    const int gain = row_end[b] - before(row_end, b);
    const bool gives = given[b] > before(given, b);
    // a sequence shrinks within its last page without giving one back: granted if it fits
    int end = ctx[b] + gain;
    if (gain == 0) {
      const long long c = static_cast<long long>(ctx[b]) + a.change[b];
      const bool ok = state_ok && ctx[b] >= 0 && ctx[b] <= cap && c >= 0 && c < ctx[b];
      if (ok && (gives || pages_of(static_cast<int>(c)) == pages_of(ctx[b]))) end = static_cast<int>(c);
    }
    a.ctx_out[b] = end;
    a.offsets[b + 1] = row_end[b];
  }
  if (leads && tid == 0) {
    a.offsets[0] = 0;
    a.state_out[0] = state_ok ? place_in_queue(pages_taken) : head;
    a.state_out[1] = state_ok ? count - pages_taken + pages_given : count;
  }
}

}  // namespace

int launch_kv4_plan(const Kv4Plan& r, cudaStream_t st) {
  PlanArgs a{};
  a.ctx = r.ctx; a.change = r.change; a.state = r.state; a.place = r.place;
  a.table = r.table; a.queue = r.queue; a.ctx_out = r.ctx_out; a.state_out = r.state_out;
  a.offsets = r.offsets; a.positions = r.positions; a.slots = r.slots;
  a.B = r.B; a.width = r.width; a.num_pages = r.num_pages; a.capacity = r.capacity; a.G = r.G; a.rows = r.rows;
  while ((1 << a.page_shift) < r.page_size) ++a.page_shift;
  a.err = device_error_word();
  if (a.err == nullptr) return fail(DFLASH2_ERR_CUDA, "no device error word");
  static unsigned done = 0;
  if (!ensure_smem_attr(kv4_plan_kernel, kPlanMaxSequences * 16, &done))
    return fail(DFLASH2_ERR_CUDA, "cudaFuncSetAttribute failed (plan)");
  // One CTA up to four rows a thread (64 sequences of 16 rows: 5.4 us, on a cluster 5.7); a cluster above, each CTA with
  // sums of its own (98304 packed rows 11 us, on one CTA 44; 4096 sequences of a row 11 and 22; each pair side by side).
  const int64_t rows = r.place != nullptr ? static_cast<int64_t>(r.B) * r.G : r.rows;
  const unsigned ctas = rows + r.B > 4 * kPlanThreads ? kPlanCluster : 1;
  cudaLaunchAttribute cl{};
  cl.id = cudaLaunchAttributeClusterDimension;
  cl.val.clusterDim.x = ctas;
  cl.val.clusterDim.y = 1;
  cl.val.clusterDim.z = 1;
  const cudaError_t e = launch_pdl(kv4_plan_kernel, dim3(ctas), dim3(kPlanThreads), static_cast<size_t>(r.B) * 16, st, &cl, 1, a);
  return e == cudaSuccess ? DFLASH2_OK : fail(DFLASH2_ERR_CUDA, "plan launch failed: %s", cudaGetErrorString(e));
}

}  // namespace dfl
