// Attention over the 4-bit key/value cache on the tcgen05 tensor cores (dflash2.ts #block: the block's queries
// attend to the context's keys and values and, bidirectionally, to the block's own).
//
// One sequence: key i < L is cached row i, key L + j its own row j (unquantised, N of them, or none); query
// row t stands at position p_t = L + N - G + t and sees key i if i < L + N, and i <= p_t (causal), and
// i > p_t - window (window > 0);
//   out_t = sum_i softmax_i(scale q_t . k_i) v_i over the keys it sees, 0 if it sees none.
//
// One CTA works on one (sequence, key/value head) and up to 80 query rows at a time, over tiles of 128
// keys. Keys are the tensor core's 128-row side in both products, so nothing is padded but the rows
// (to N, a multiple of 16):
//   S^T [128 keys x N rows]   = K tile [keys][D] . Q [rows][D]^T         (K-major operands)
//   O^T [D channels x N rows] += V tile [keys][D]^T . P^T [keys][rows]   (both MN-major: V as it lies)
// A softmax thread holds one key's scores of all (half of the) rows. It needs no reduction over keys:
// the rows' reference (the number subtracted before the exponential) is only raised when some number
// passes it by 2^8, which all threads agree on by one barrier a tile; then, rarely and once a tile, the
// rows' maxima are taken, and O and the sums rescaled. The sums stay per thread until the end.
//
// Precision: operands are fp16 (11 significant bits; with bf16 the keys', the values' and the
// probabilities' roundings add up to twice the rounding of the bf16 result). fp16's range does not hold
// every bf16 value, so each key row and each value row is divided by a power of two that brings its
// largest value to [1, 2), and Q by one for all rows (one a row where rows differ by more than 2^14). Cached
// rows go to 2^-7 of that, for scale 2^24 to fit (dequant_word): their channels more than 2^7 below the row's
// largest have steps of 2^-17 of it (6 bits are left of a group 2^12 below the row's other). The keys'
// factor multiplies the thread's scores, and the values' is added to them as its logarithm (one FMA): the
// operand P holds probabilities times values' factors over the row's own largest such product, so that a
// value row far larger than the rest counts in the rows that give it weight and is not felt by those that do
// not, to which a mask may hide it. The sums take the factor off again, in fp32.
//
// Warps: 8 softmax (two per 32 TMEM lanes, half of the rows each), 8 dequant (four for K, four for V, 32
// keys of a tile each: codes -> fp16 operand tiles in shared memory, 128-byte swizzle), 2 MMA (one elected
// thread each for S and for O: an MMA takes some 20 cycles to issue, and 100 from a thread picked by its number, for
// which descriptors do not stay in uniform registers: 32 trees of 32 rows 162 us instead of 147), 2 copy (a ring of bulk
// copies for K, one for V). K, V and S are double-buffered. The softmax warps, whose sums stay in registers,
// take some of the others' (kSoftRegs).
//
// What a tile takes: 2.3 to 2.5 thousand cycles with 80 rows, where the softmax warps' chain (scores from TMEM,
// the check, exponentials, the operand's stores and their fence) is the longest, and 1.9 with 16, where the
// conversion of codes is; each scheduler issues in 49 % and 57 % of the cycles. 64 blocks of 16 rows and five
// query heads a key head over 256 to 4096 keys of 128 channels take 125 us, 64 single tokens over 1 to 8192 keys 112 us
// (2.7 TB/s of the cache). What was slower (each against the code of its time): sixteen softmax warps; two sets of dequant warps taking tiles in
// turn (118 us for the tokens); K converted into TMEM (155 us: the loops then miss the instruction cache); the
// check split into an arrival and a later wait (172 us for the blocks); the next tile's codes read ahead (126 us); the
// scores' buffer given back together with the operand (130 us for the tokens).
//
// Trees: a row's own keys are its line of ancestors, 64 bits that the own tile's masks are taken from; all else is the
// same code. 32 trees of 32 rows (160 rows a key head) over 256 to 4096 keys take 140 us (131 to 149 by the lengths drawn, 62
// to 79 thousand keys in all), one of 64 rows over 32768 keys 87: the same chain a tile, for which shared memory moves 224
// KB (operands into the products 104, their making 64), 1.7 of its thousand cycles at 128 bytes a clock. One of 8 rows over 1024 keys takes 17 us: start 4, three tiles and the join.
//
// CTAs are persistent, one an SM: all (sequence, head, row tile) items, each its tiles and a constant for
// the change from one item to the next, form one line that is cut into equal ranges, whatever the lengths.
// An item that spans several ranges is finished by the range that holds its last tile: the earlier ones
// leave partial results in the workspace and raise a flag there. Up to eight parts are joined by the last
// range; of more, groups of about their number's square root are joined by the last range of each, and then
// the groups. (So results do not depend on timing, and a range waits only for CTAs dispatched before it.) A
// flag holds the call's own 64-bit number, so the workspace needs no initialisation, and its reader clears it
// for a replay. A block over 32768 keys, 19 parts a head, takes 42 us of which the joins are 12; a kernel of
// its own for them took 20.
//
// A CTA leaves only when everything that arrives on its barriers by itself has arrived: the copies by those who wait for them,
// the products' releases by their issuers (await_releases).
//
// No wait blocks for ever, no loop but over tiles, parts and rows, and no wait is skipped: after a timeout the
// roles run on (their results are void and the error word says so), so that every barrier stays balanced.
#include <algorithm>

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

template <int D, int NK>                    // N = 16 NK rows
struct BlockCfg {
  static constexpr int N = 16 * NK;
  // the change from one item to the next, in tiles (measured: 15 of 3.1 thousand cycles with 80 rows, 5 of
  // 2.0 with 16). A tree's has its lines of ancestors and the masks of its own rows besides, and a row tile of it takes
  // 19 of 2.2 thousand cycles longer than its tiles: 32 trees of 32 rows over 256 to 4096 keys take 147 us with 5 there, 130
  // with 9 and 134 with 12 (one draw of lengths); of 4 rows (NK = 2) 46 with 3, 44 with 4.
  static constexpr int setup(bool tree) { return NK <= 2 ? (tree ? 4 : 3) : (tree ? NK + 4 : NK); }
  // registers a thread: 640 x 96 at launch, then shared out. With 80 rows 144 / 64 takes 128 to 130 us for 64
  // blocks over 256 .. 4096 keys where 120 / 80 takes 147, 136 / 64 133 and 152 / 56 132; with 16 rows, whose softmax
  // threads need few, 120 / 80 takes 111 us for 64 tokens over 1 .. 8192 keys and 152 / 56 128.
  static constexpr int kSoftRegs = NK >= 4 ? 144 : 120, kOtherRegs = NK >= 4 ? 64 : 80;
  static_assert(kBSoft * kSoftRegs + (kBThreads - kBSoft) * kOtherRegs <= kBThreads * 96, "registers");
  static constexpr int kHalves = D / 64;                     // 64-channel halves of a K or V tile
  static constexpr int kTileBytes = kHalves * kBTile * 128;  // fp16 [half][key][64]
  static constexpr int kPBytes = (N > 64 ? 2 : 1) * kBTile * 128;
  static constexpr int kQBytes = kHalves * N * 128;
  static constexpr int kOffV = 2 * kTileBytes;
  static constexpr int kOffP = kOffV + 2 * kTileBytes;  // (D = 64: the MMA reads one half past V: P)
  static constexpr int kOffQ = kOffP + kPBytes;
  static constexpr int kRaw = kBTile / kKvGranule * KvLayout<D>::kGranuleBytes;  // a tile of one side: [granule]
  static constexpr int kRawStages = NK == 5 ? 2 : 3;
  static constexpr int kOffRaw = kOffQ + kQBytes;            // [side][stage]
  static constexpr int kOffInfo = kOffRaw + 2 * kRawStages * kRaw;           // float2 [4][128]: key factor, value factor
  static constexpr int kOffRow = kOffInfo + 4 * kBTile * 8;  // per row: t, lo, hi, factor, offset, query factor
  static constexpr int kOffSum = kOffRow + 6 * N * 4;        // float [4][N]
  static constexpr int kOffBar = (kOffSum + 4 * N * 4 + 15) / 16 * 16;
  static constexpr int kOffTree = kOffBar + 384;             // (trees) uint32 [2][N]: the own rows that each row sees
  static constexpr int kSmem = 1024 + kOffTree, kSmemTree = kSmem + 2 * N * 4 + kTreeRows * 8;  // and uint64 [64]: lines
  static constexpr uint32_t kTmemCols = 3 * N <= 64 ? 64 : (3 * N <= 128 ? 128 : (3 * N <= 256 ? 256 : 512));
};

struct BlockArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const uint8_t* cache;
  const int32_t *table, *ctx;  // (read by ordinary loads: the kernel in front may write them while this one starts)
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
__device__ __forceinline__ bool bar_or(bool p) {  // over the softmax threads
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(p)), "n"(kBSoft)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_soft() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kBSoft) : "memory"); }

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

__device__ __forceinline__ void tmem_ld8(uint32_t t, float* x) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const float* x) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(x);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// (Suspended, not spinning: the issue slots belong to the warps that work. Lanes may part here and in votes: what the whole
// warp has to execute together, as tensor memory's loads and waits, comes behind a __syncwarp.)
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
// The last releases of two buffers that took `tiles` tiles in turn: no role waits for those, and a CTA must not leave
// before they have arrived on its barriers. (Tile i completes phase i / 2 of buffer i % 2.)
__device__ __forceinline__ void await_releases(uint32_t empty, uint32_t tiles, volatile int* abort_flag, int* err) {
  for (uint32_t i = tiles - min(tiles, 2u); i < tiles; ++i) wait_on(empty + 8 * (i & 1u), (i >> 1) & 1u, abort_flag, err);
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
  s.L = min(max(a.ctx[b], 0), a.cap);  // (block_range records a length outside)
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
    const int len = a.ctx[b];
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

// Eight values reduced over a warp's lanes, halving the values a lane carries with each step: afterwards the
// lanes 4 m .. 4 m + 3 hold value warp_reduce8_row.
template <typename F>
__device__ __forceinline__ float warp_reduce8(const float* x, int lane, F op) {
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float give = (lane & 16) ? x[i] : x[4 + i];
    s[i] = op((lane & 16) ? x[4 + i] : x[i], __shfl_xor_sync(0xffffffffu, give, 16));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float give = (lane & 8) ? s[i] : s[2 + i];
    s[i] = op((lane & 8) ? s[2 + i] : s[i], __shfl_xor_sync(0xffffffffu, give, 8));
  }
  const float give = (lane & 4) ? s[0] : s[1];
  float v = op((lane & 4) ? s[1] : s[0], __shfl_xor_sync(0xffffffffu, give, 4));
  v = op(v, __shfl_xor_sync(0xffffffffu, v, 2));
  return op(v, __shfl_xor_sync(0xffffffffu, v, 1));
}
__device__ __forceinline__ int warp_reduce8_row(int lane) {
  return ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
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

// The item of a range's first piece, if earlier ranges began it, and what the range does for it.
struct BlockJoin {
  long long start;
  int b, head, rt, tiles;
  bool ends, leads;  // its last tile lies here; a group of its parts ends here
};

// Joins the parts of an item, or of a group: the softmax threads. The parts come into the operands' place (the
// products are done) by bulk copies, three in flight: an SM reads 64 bytes a clock from L2.
template <int D, int NK, bool kTree>
__device__ __forceinline__ void block_join(const BlockArgs& a, const BlockLine& line, const BlockJoin& j, uint8_t* smem,
                                           uint32_t full, volatile int* abort_flag) {
  using C = BlockCfg<D, NK>;
  constexpr int N = C::N, kSlot = N * D * 4, kItems = N * D / 4 / kBSoft;
  static_assert(3 * kSlot <= 4 * C::kTileBytes, "the parts' place");
  const int me = static_cast<int>(blockIdx.x);
  const BlockParts parts(line, j.start, C::setup(kTree), j.tiles);
  const int head = j.head, row_first = j.rt * a.tile_rows;
  const int nrows = min(a.tile_rows, a.rows - row_first), count = parts.inputs(me);
  // the parts' maxima and sums, then their weights, per row; at most 25 of 169 CTAs
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffP);       // [count][N]
  int* place = reinterpret_cast<int*>(smem + C::kOffInfo);       // [count]: the parts' slots
  float* row_f = reinterpret_cast<float*>(smem + C::kOffRow);    // [N]
  static_assert(25 * N * 8 <= C::kPBytes, "the parts' weights");
  if (threadIdx.x < count) {
    const int c = parts.input(me, threadIdx.x);
    place[threadIdx.x] = parts.slot(c);
    if (c != me) {
      unsigned long long* flag = a.flags + c;
      const uint64_t t0 = globaltimer_ns();
      while (ld_acquire_u64(flag) != a.call) {
        __nanosleep(64);
        if (*abort_flag != 0 || globaltimer_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1;
          atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_TIMEOUT));
          break;
        }
      }
      *flag = 0ull;  // read: ready for a replay
    }
  }
  bar_soft();
  const uint32_t bytes = static_cast<uint32_t>(nrows * D * 4);
  auto fetch = [&](int p) {  // part p into its place
    const uint32_t bar = full + 8 * (p % 3);
    mbar_arrive_expect_tx(bar, bytes);
    bulk_load(smem_u32(smem) + (p % 3) * kSlot, a.part_o + static_cast<int64_t>(place[p]) * N * D, bytes, bar);
  };
  if (threadIdx.x == 0) {
    fence_proxy_async_all();  // (written by other CTAs' plain stores, read by the copy engine)
    for (int p = 0; p < min(3, count); ++p) fetch(p);
  }
#pragma unroll 1
  for (int p = threadIdx.x >> 5; p < count; p += kBSoftWarps)
    for (int r = threadIdx.x & 31; r < nrows; r += 32)
      ml[p * N + r] = __ldcg(a.part_ml + static_cast<int64_t>(place[p]) * N + r);
  bar_soft();
  if (threadIdx.x < nrows) {
    float2* mine = ml + threadIdx.x;
    float mm = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int p = 0; p < count; ++p) mm = fmaxf(mm, mine[p * N].x);
#pragma unroll 1
    for (int p = 0; p < count; ++p) {
      const float2 v = mine[p * N];
      const float f = v.x == -INFINITY ? 0.f : ex2_approx(v.x - mm);
      sum += f * v.y;
      mine[p * N].x = f;
    }
    if (j.leads) __stcg(a.part_ml + static_cast<int64_t>(place[count - 1]) * N + threadIdx.x, make_float2(mm, sum));
    row_f[threadIdx.x] = j.leads ? 1.f : (sum == 0.f ? 0.f : kBSumUnit / sum);  // (NaN stays)
  }
  bar_soft();
  float4 acc[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kRowStep = kBSoft / (D / 4);
  const int r0 = threadIdx.x / (D / 4), col = threadIdx.x % (D / 4) * 4;
#pragma unroll 1
  for (int p = 0; p < count; ++p) {
    wait_on(full + 8 * (p % 3), static_cast<uint32_t>(p / 3) & 1u, abort_flag, a.err);
    const float* from = reinterpret_cast<const float*>(smem + (p % 3) * kSlot) + r0 * D + col;
    const float2* weight = ml + p * N + r0;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const float f = weight[k * kRowStep].x;
      const float4 v = *reinterpret_cast<const float4*>(from + k * kRowStep * D);
      if (r0 + k * kRowStep < nrows && f != 0.f) {  // (0: nothing of the row there)
        acc[k].x += f * v.x; acc[k].y += f * v.y; acc[k].z += f * v.z; acc[k].w += f * v.w;
      }
    }
    bar_soft();
    if (threadIdx.x == 0 && p + 3 < count) fetch(p + 3);
  }
  float* part = a.part_o + static_cast<int64_t>(place[count - 1]) * N * D;
  __nv_bfloat16* out = a.out + static_cast<int64_t>(j.b) * a.G * a.Hq * D + head * a.R * D + col;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int r = r0 + k * kRowStep;
    if (r >= nrows) break;
    if (j.leads) {
      __stcg(reinterpret_cast<float4*>(part + r * D + col), acc[k]);
    } else {
      const float inv = row_f[r];
      const int rr = row_first + r, t = row_token(a, rr);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[k].x * inv, acc[k].y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[k].z * inv, acc[k].w * inv);
      uint2 u;
      u.x = *reinterpret_cast<const uint32_t*>(&lo);
      u.y = *reinterpret_cast<const uint32_t*>(&hi);
      *reinterpret_cast<uint2*>(out + static_cast<int64_t>(t * a.Hq + rr - t * a.R) * D) = u;
    }
  }
}

// kTree: the block's rows are a tree's. Row t stands at position L + (its ancestors' number) and sees, of the block's
// own rows, its ancestors and itself.
template <int D, int NK, bool kTree>
__global__ void __launch_bounds__(kBThreads, 1) kv4_attention_kernel(const BlockArgs a) {
  using C = BlockCfg<D, NK>;
  using L = KvLayout<D>;
  constexpr int kSetup = C::setup(kTree);
  using Walk = BlockWalk<kSetup>;
  constexpr int N = C::N, NH = N / 2;  // rows, a softmax thread's rows
  constexpr int NCH = D / 32;   // 32-channel chunks of a row
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  float2* info = reinterpret_cast<float2*>(smem + C::kOffInfo);      // [4][128]
  float* row_t = reinterpret_cast<float*>(smem + C::kOffRow);        // minus the reference
  int* row_lo = reinterpret_cast<int*>(row_t + N);                   // keys [lo, hi) that the row sees
  int* row_hi = row_lo + N;
  float* row_f = reinterpret_cast<float*>(row_hi + N);               // what the row's sum and O shrink by; at the end, O's factor
  int* row_off = reinterpret_cast<int*>(row_f + N);                  // where the row starts in the sequence's out
  float* row_q = reinterpret_cast<float*>(row_off + N);              // what the query row's scores are multiplied by
  float* row_red = reinterpret_cast<float*>(smem + C::kOffSum);      // [4][N] the TMEM quarters' maxima or sums
  // barriers, as shared addresses
  const uint32_t bars = smem_u32(smem + C::kOffBar);
  const uint32_t kfull = bars, kempty = bars + 16, vfull = bars + 32, vempty = bars + 48;     // [2] each
  const uint32_t sfull = bars + 64, sempty = bars + 80, pfull = bars + 96, odone = bars + 104, qfull = bars + 112;
  const uint32_t raw_full = bars + 120, raw_empty = bars + 168;                               // [side][3]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 216);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* qmax = tmem_slot + 2;
  uint32_t* qmin = tmem_slot + 3;
  volatile int* mixed = reinterpret_cast<volatile int*>(tmem_slot + 4);
  uint32_t* came_s = tmem_slot + 5;  // [side][3]: the granules that came
  const uint32_t join_full = bars + 264;  // [3]
  uint32_t* row_tree = reinterpret_cast<uint32_t*>(smem + C::kOffTree);        // [2][N]
  uint64_t* tree_line = reinterpret_cast<uint64_t*>(row_tree + 2 * N);         // [64]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull + 8 * i, kBDeqWarps / 2);
      mbar_init(vfull + 8 * i, kBDeqWarps / 2);
      mbar_init(kempty + 8 * i, 1);
      mbar_init(vempty + 8 * i, 1);
      mbar_init(sfull + 8 * i, 1);
      mbar_init(sempty + 8 * i, kBSoftWarps);
    }
    mbar_init(pfull, kBSoftWarps);
    mbar_init(odone, 1);
    for (int i = 0; i < 3; ++i) mbar_init(join_full + 8 * i, 1);
    mbar_init(qfull, kBSoftWarps);
    for (int i = 0; i < 6; ++i) {
      mbar_init(raw_full + 8 * i, 1);
      mbar_init(raw_empty + 8 * i, kBDeqWarps / 2);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kBMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();
  const BlockRange range = block_range(a, kSetup, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));

  if (warp >= kBSoftWarps && warp < kBSoftWarps + kBDeqWarps) {
    // ------------------------------------------------------------------ dequant
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    const int side = (warp - kBSoftWarps) >> 2, dw = warp & 3;  // K or V; keys 32 dw .. of each tile
    const uint32_t low = side == 0 ? kBPow2Low : kBPow2LowQV;
    const int ch = lane % NCH;
    constexpr int kStep = 32 / NCH;                        // step i converts keys sub + i kStep of the warp's 32
    const int sub = lane / NCH;
    const uint8_t* ring = smem + C::kOffRaw + side * C::kRawStages * C::kRaw + dw * 2 * L::kGranuleBytes;
    const uint32_t rfull = raw_full + side * 24, rempty = raw_empty + side * 24;
    const uint32_t full = side == 0 ? kfull : vfull, empty = side == 0 ? kempty : vempty;
    // where the lane's four 16-byte pieces of its first key go (key & 7 is the same in every step)
    uint32_t to[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int pc = piece_of_word<D>(ch * 4 + k);
      to[k] = smem_u32(smem) + side * C::kOffV + (pc >> 3) * (kBTile * 128) + (dw * 32 + sub) * 128 +
              (((pc & 7) ^ (sub & 7)) << 4);
    }
    const uint8_t* codes0 = ring + sub * L::kRow + ch * 16;
    const uint8_t* par0 = ring + (lane >> 4) * L::kGranuleBytes + L::kCodes + (lane & 15) * L::kGroups * 4;
    uint32_t it = 0, stage = 0, rphase = 0;
    for (Walk w(a, range); w.valid(); w.next(a)) {
      const __nv_bfloat16* own_src = (side == 0 ? a.k_new : a.v_new);
      if (own_src != nullptr) {
        own_src += static_cast<int64_t>(w.b) * a.G * a.new_stride + w.head * D;
        if (w.j1 > w.seq.cached && dw * 32 + lane < a.G)  // the piece ends with its own rows
#pragma unroll
          for (int x = 0; x < D; x += 64) prefetch_l1(own_src + (dw * 32 + lane) * a.new_stride + x);
      }
      // the lane's key of the piece's tile j is seen for 128 j in [seen_lo, seen_hi)
      const int at = (w.seq.lo & ~(kBTile - 1)) + dw * 32 + lane;
      const int seen_lo = w.seq.lo - at, seen_hi = w.seq.hi - at;
#pragma unroll 1
      for (int j = w.j0; j < w.j1; ++j, ++it) {
        const uint32_t buf = it & 1u;
        const uint32_t par = ((it >> 1) & 1u) ^ 1u;
        const uint32_t tile = buf * C::kTileBytes;
        // the factors travel in a ring of four: tile it - 4's were read before tile it - 2's operands were
        // released, which `empty` reports
        float* inf = reinterpret_cast<float*>(info + (it & 3u) * kBTile + dw * 32) + side;
        const bool cached = j < w.seq.cached;
        if (cached || own_src == nullptr) {
          // 32 keys from the ring. Rows that no query sees may hold anything: they count as zeros.
          bool in = false;  // (neither cached nor own: a tile without keys)
          if (cached) {
            wait_on(rfull + 8 * stage, rphase, abort_flag, a.err);
            in = ((came_s[side * 3 + stage] >> (2 * dw + (lane >> 4))) & 1u) && j * kBTile >= seen_lo && j * kBTile < seen_hi;
          }
          const uint32_t raw = stage * C::kRaw;
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
          const float f = odd ? __uint_as_float(0x7fffffffu) : row_params<L::kGroups>(pr, po, low);
          uint32_t sb_bits[NCH];
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            const uint32_t w0 = __shfl_sync(0xffffffffu, po[0], sub + i * kStep);
            const uint32_t w1 = L::kGroups == 2 ? __shfl_sync(0xffffffffu, po[1], sub + i * kStep) : w0;
            sb_bits[i] = ch >= 2 ? w1 : w0;
          }
          if (cached) {  // read out: every lane's loads come before the arrival
            __syncwarp();
            if (lane == 0) mbar_arrive(rempty + 8 * stage);
            if (++stage == C::kRawStages) {
              stage = 0;
              rphase ^= 1u;
            }
          }
          wait_on(empty + 8 * buf, par, abort_flag, a.err);
          inf[2 * lane] = side == 0 || in ? f : -1.f;  // values' -1: the key is not there
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
              const bool odd = side == 1 && m >= kBInfinity;  // (as for cached rows)
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
  } else if (warp >= kBMmaWarp) {
    // (a warpgroup, four warps, gives its registers up by one instruction that it executes together)
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp < kBCopyWarp) {
      // ------------------------------------------------------------------ MMA issuers: S, and O
      if (elect_one()) {
        constexpr uint32_t kFmt = (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);  // f32 <- f16, M = 128
        uint32_t it = 0, piece = 0;
        // descriptors: the lower words of the operands' first steps (address / 16, leading offset), and the
        // upper word (stride 1024 bytes, 128-byte swizzle), the same for all
        if (warp == kBMmaWarp) {
          const uint64_t kd = desc_kmajor_sw128(smem_u32(smem)), qd = desc_kmajor_sw128(smem_u32(smem + C::kOffQ));
          const uint32_t hi = static_cast<uint32_t>(kd >> 32), k_lo = static_cast<uint32_t>(kd), q = static_cast<uint32_t>(qd);
          for (Walk w(a, range); w.valid(); w.next(a), ++piece) {
            wait_on(qfull, piece & 1u, abort_flag, a.err);
#pragma unroll 1
            for (int j = w.j0; j < w.j1; ++j, ++it) {
              const uint32_t buf = it & 1u;
              wait_on(sempty + 8 * buf, ((it >> 1) & 1u) ^ 1u, abort_flag, a.err);
              wait_on(kfull + 8 * buf, (it >> 1) & 1u, abort_flag, a.err);
              tc_fence_after();
              const uint32_t k = k_lo + buf * (C::kTileBytes / 16), d = tmem + buf * N;
              mma_lean<true>(d, k, q, hi, hi, kFmt);
#pragma unroll
              for (int s = 1; s < D / 16; ++s)
                mma_lean<false>(d, k + (s >> 2) * (kBTile * 128 / 16) + 2 * (s & 3), q + (s >> 2) * (N * 128 / 16) + 2 * (s & 3),
                                hi, hi, kFmt);
              mma_commit(sfull + 8 * buf);
              mma_commit(kempty + 8 * buf);
            }
          }
          await_releases(kempty, it, abort_flag, a.err);
        } else {
          const uint64_t vd = desc_keys_sw128(smem_u32(smem + C::kOffV)), pd = desc_keys_sw128(smem_u32(smem + C::kOffP));
          const uint32_t hi = static_cast<uint32_t>(vd >> 32), v_lo = static_cast<uint32_t>(vd), p = static_cast<uint32_t>(pd);
          constexpr uint32_t id = kFmt | (1u << 15) | (1u << 16);
          const uint32_t d = tmem + 2 * N;
          for (Walk w(a, range); w.valid(); w.next(a))
#pragma unroll 1
            for (int j = w.j0; j < w.j1; ++j, ++it) {
              const uint32_t buf = it & 1u;
              wait_on(vfull + 8 * buf, (it >> 1) & 1u, abort_flag, a.err);
              wait_on(pfull, it & 1u, abort_flag, a.err);
              tc_fence_after();
              const uint32_t v = v_lo + buf * (C::kTileBytes / 16);
              if (j > w.j0)
                mma_lean<false>(d, v, p, hi, hi, id);
              else
                mma_lean<true>(d, v, p, hi, hi, id);
#pragma unroll
              for (int s = 1; s < kBTile / 16; ++s) mma_lean<false>(d, v + 128 * s, p + 128 * s, hi, hi, id);
              mma_commit(odone);
              mma_commit(vempty + 8 * buf);
            }
          await_releases(vempty, it, abort_flag, a.err);
        }
        if (*abort_flag != 0) {  // the MMAs in flight end before the CTA leaves
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 2000000ull) {
          }
        }
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ copies of one side
      // A lane per granule looks up its page; the first granule of each run that lies together in a page
      // (the tile, a page, or a granule) is copied with the rest of its run.
      const int side = warp - kBCopyWarp;
      const int granules = (1 << a.page_shift) / kKvGranule, run = min(granules, kBTile / kKvGranule);
      const uint32_t rfull = raw_full + side * 24, rempty = raw_empty + side * 24;
      uint32_t stage = 0, phase = 1;
      for (Walk w(a, range); w.valid(); w.next(a)) {
        const int last = min(w.j1, w.seq.cached);
        for (int j0 = w.j0; j0 < last; j0 += 4) {  // pages of four tiles at a time: 32 granules
          const int g0 = ((w.seq.lo >> kBTileLog) + j0) * (kBTile / kKvGranule) + lane;  // the lane's granule of the sequence
          const int key = g0 * kKvGranule;
          int page = -1;
          // a granule that some row sees (a window may have left the others' pages behind)
          if (j0 + lane / 8 < last && key < w.seq.hi && key + kKvGranule > w.seq.lo) {
            page = a.table[static_cast<int64_t>(w.b) * a.width + (key >> a.page_shift)];
            if (page < 0 || page >= a.num_pages) {
              atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_BAD_INDEX));
              page = -1;
            }
          }
          const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
          for (int j = j0; j < min(j0 + 4, last); ++j) {
            const uint32_t got = (have >> (8 * (j - j0))) & 0xffu;
            wait_on(rempty + 8 * stage, phase, abort_flag, a.err);
            if (lane == 0) {
              came_s[side * 3 + stage] = got;
              mbar_arrive_expect_tx(rfull + 8 * stage, static_cast<uint32_t>(__popc(got)) * L::kGranuleBytes);
            }
            __syncwarp();
            const int g = lane & 7, first = g & ~(run - 1);
            // the granules of this lane's run that came, copied by the lane of the first of them (those no
            // row sees lie at the run's ends, so what came is contiguous)
            const uint32_t mine = (got >> first) & ((1u << run) - 1u);
            if (lane / 8 == j - j0 && mine != 0u && g == first + __ffs(mine) - 1)
              bulk_load(smem_u32(smem + C::kOffRaw + (side * C::kRawStages + stage) * C::kRaw + g * L::kGranuleBytes),
                        a.cache + (((static_cast<int64_t>(page) * a.Hkv + w.head) * 2 + side) * granules +
                                   (g0 & (granules - 1))) *
                                      static_cast<int64_t>(L::kGranuleBytes),
                        static_cast<uint32_t>(__popc(mine)) * L::kGranuleBytes, rfull + 8 * stage);
            __syncwarp();
            if (++stage == C::kRawStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    __syncwarp();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    const int quad = warp & 3;                    // TMEM lanes 32 quad .., rows (warp / 4) NH ..
    const int key_in = quad * 32 + lane;          // the thread's key of each tile; at the end, its channel
    const int r0 = (warp >> 2) * NH;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(r0);
    uint32_t to[NK];                              // where eight rows' probabilities of the thread's key go
#pragma unroll
    for (int c = 0; c < NK; ++c) {
      const int r8 = r0 / 8 + c;
      to[c] = smem_u32(smem + C::kOffP) + key_in * 128 + (r8 >> 3) * (kBTile * 128) + (((r8 & 7) ^ (key_in & 7)) << 4);
    }
    // Q of a piece: its rows as fp16, channels in the codes' order, over a power of two common to all (returned),
    // with which rows 2^14 smaller than the largest still have 11 significant bits. Where some channels lie
    // further below it, or are not finite, each row goes over its own power (`mixed`), and row_q multiplies its
    // scores: where references are raised, so that the piece's every tile goes there. A row that is not finite
    // becomes NaN, and does not count for the others.
    auto load_q = [&](const Walk& w) {
      const int head = w.head, row_first = w.rt * a.tile_rows;
      const int nrows = min(a.tile_rows, a.rows - row_first);
      constexpr int kQItems = (N * (D / 8) + kBSoft - 1) / kBSoft;
      auto fetch = [&](int r, int c) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < nrows) {
          const int rr = row_first + r, t = row_token(a, rr);
          v = __ldg(reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(w.b) * a.G + t) * a.q_stride +
                                                   (head * a.R + rr - t * a.R) * D + 8 * c));
        }
        return v;
      };
      auto store = [&](int r, int c, const uint4& v) {
        const int pc = piece_of_word<D>(c);
        *reinterpret_cast<uint4*>(smem + C::kOffQ + (pc >> 3) * (N * 128) + r * 128 + (((pc & 7) ^ (r & 7)) << 4)) = v;
      };
      uint4 qv[kQItems];
#pragma unroll
      for (int i = 0; i < kQItems; ++i) {
        const int x = threadIdx.x + i * kBSoft;
        qv[i] = fetch(x / (D / 8), x % (D / 8));
      }
      if (threadIdx.x == 0) {
        *qmax = 0u;
        *qmin = kBInfinity;
      }
      bar_soft();
      uint32_t most = 0, least = kBInfinity;
#pragma unroll
      for (int i = 0; i < kQItems; ++i) {
        const uint32_t m = max_abs8(qv[i]);
        most = max(most, m);
        least = min(least, m - 1u);  // (zeros do not count)
      }
      most = __reduce_max_sync(0xffffffffu, most);
      least = __reduce_min_sync(0xffffffffu, least);
      if (lane == 0) {
        atomicMax(qmax, most);
        atomicMin(qmin, least);
      }
      if (threadIdx.x < N) row_q[threadIdx.x] = 1.f;
      bar_soft();
      most = *qmax;
      const float common = pow2_of(__uint_as_float(most), kBPow2LowQV);
      const bool mix = most >= kBInfinity || pow2_of(__uint_as_float(*qmin), kBPow2LowQV) * kBLiftQ < common;
      if (threadIdx.x == 0) *mixed = mix ? 1 : 0;
      if (!mix) {
#pragma unroll
        for (int i = 0; i < kQItems; ++i) {
          const int x = threadIdx.x + i * kBSoft;
          if (x / (D / 8) < N) store(x / (D / 8), x % (D / 8), convert_word(qv[i], pow2_inverse(common) * kBLiftQ));
        }
      } else {
#pragma unroll 1
        for (int x = threadIdx.x; x < (N * (D / 8) + 31) / 32 * 32; x += kBSoft) {  // whole warps
          const int r = x / (D / 8), c = x % (D / 8);
          const uint4 v = fetch(r, c);
          uint32_t m = max_abs8(v);
#pragma unroll 1
          for (int k = 1; k < D / 8; k <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
          const float own = pow2_of(__uint_as_float(m), kBPow2LowQV);
          if (r < N) {
            store(r, c, m < kBInfinity ? convert_word(v, pow2_inverse(own) * kBLiftQ)
                                       : make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu));
            if (c == 0) row_q[r] = own * (1.f / kBLiftQ);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
      return mix ? 1.f : common * (1.f / kBLiftQ);
    };
    uint32_t it = 0;
    Walk w(a, range);
    bool gave = false;  // the last piece goes on in the next range
    int tree_of = -1;   // the sequence whose lines of ancestors are in shared memory
    BlockJoin join{w.start, w.b, w.head, w.rt, w.seq.tiles, w.valid() && w.j0 > 0 && w.j1 == w.seq.tiles, false};
    Walk next = w;
    for (bool first = true;; first = false) {
      float qf = 1.f;
      if (next.valid()) qf = load_q(next);  // (every S of the piece before is done): its scores start meanwhile
      if (!first) {
        // ---- the result of the item before (or of its part)
        const int row_first = w.rt * a.tile_rows, nrows = min(a.tile_rows, a.rows - row_first);
        const bool complete = w.j0 == 0 && w.j1 == w.seq.tiles;
        bar_soft();
        const int64_t slot = (static_cast<int64_t>(blockIdx.x) * 2 + (w.j0 > 0 ? 0 : 1)) * N;
        if (threadIdx.x < N) {
          const int r = threadIdx.x;
          float sum = row_red[r] + row_red[N + r] + row_red[2 * N + r] + row_red[3 * N + r];
          if (kTree && row_t[r] == kBPadding) sum = 0.f;  // (whatever a row that is not there holds)
          // (a row that saw something that is not finite has a sum, and an O, of NaN)
          row_f[r] = sum == 0.f ? 0.f : (complete ? kBSumUnit / sum : 1.f);
          if (!complete && r < nrows) a.part_ml[slot + r] = make_float2(row_t[r] != kBUnseen ? -row_t[r] : -INFINITY, sum);
        }
        bar_soft();
        // the thread's channel: operand position p of each eight holds channel p / 2 + 4 (p % 2) of its word
        const int ch = word_of_piece<D>(key_in >> 3) * 8 + ((key_in & 7) >> 1) + 4 * (key_in & 1);
        wait_on(odone, (it - 1) & 1u, abort_flag, a.err);
        tc_fence_after();
        __syncwarp();
        __nv_bfloat16* out = a.out + static_cast<int64_t>(w.b) * a.G * a.Hq * D + ch;
        float* part = a.part_o + (slot + r0) * D + ch;
        float o[NH];
#pragma unroll
        for (int c = 0; c < NH; c += 8) tmem_ld8(tl + static_cast<uint32_t>(2 * N + c), o + c);
        tmem_ld_wait();
        if (key_in < D) {
          const int n = nrows - r0;
#pragma unroll
          for (int r = 0; r < NH; r += 4) {
            const float4 g4 = *reinterpret_cast<const float4*>(row_f + r0 + r);
            const int4 o4 = *reinterpret_cast<const int4*>(row_off + r0 + r);
            const float g[4] = {g4.x, g4.y, g4.z, g4.w};
            const int off[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v = g[i] != 0.f ? o[r + i] * g[i] : 0.f;  // (O of a row that saw nothing is not looked at)
              if (r + i < n) {
                if (complete)
                  out[off[i]] = __float2bfloat16_rn(v);
                else
                  part[(r + i) * D] = v;
              }
            }
          }
        }
        __syncwarp();
        tc_fence_before();
        bar_soft();  // the rows' data are read before the next piece sets them
      }
      if (!next.valid()) break;
      w = next;
      const int head = w.head, row_first = w.rt * a.tile_rows;
      const int nrows = min(a.tile_rows, a.rows - row_first);
      if (kTree && w.b != tree_of) {  // each row's line of ancestors (the items of a sequence follow one another)
        tree_of = w.b;
        if (warp == 0) {
          int parent[2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            parent[i] = lane + 32 * i < a.G ? __ldg(a.parents + static_cast<int64_t>(w.b) * a.G + lane + 32 * i) : -2;
          bool bad;
          const TreeLines tree = tree_lines(parent, a.G, bad);
          if (bad) atomicCAS(a.err, 0, static_cast<int>(DFLASH2_ERR_BAD_INDEX));
          tree_line[lane] = tree.line[0];
          tree_line[lane + 32] = tree.line[1];
        }
        bar_soft();
      }
      if (threadIdx.x < N) {
        const int r = threadIdx.x, rr = row_first + r, t = row_token(a, rr);
        uint64_t line = 0;
        if (kTree && r < nrows) line = tree_line[t];
        const int pos = w.seq.base + (kTree ? __popcll(line) - 1 : t);
        const int all = w.seq.L + (a.k_new != nullptr ? a.G : 0);
        const bool there = r < nrows && (!kTree || line != 0);
        row_t[r] = there ? kBUnseen : kBPadding;
        row_lo[r] = a.window > 0 ? max(0, pos - a.window + 1) : 0;
        row_hi[r] = there ? (kTree ? w.seq.L : (a.causal ? min(all, pos + 1) : all)) : 0;
        if (kTree) {
          if (a.window > 0)
            for (int n = __popcll(line); n > a.window; --n) line &= line - 1;
          row_tree[r] = static_cast<uint32_t>(line);
          row_tree[N + r] = static_cast<uint32_t>(line >> 32);
        }
        row_off[r] = (t * a.Hq + head * a.R + rr - t * a.R) * D;
      }
      bar_soft();
      const float qscale = qf * a.scale_log2;
      // seen by every row of the tile: [all_lo, all_hi)
      const int t_first = row_token(a, row_first), t_last = row_token(a, row_first + nrows - 1);
      const int all_lo = a.window > 0 ? w.seq.base + t_last - a.window + 1 : 0;
      const int all_hi = a.causal ? w.seq.base + t_first + 1 : 0x7fffffff;

      float l[NH];
#pragma unroll
      for (int r = 0; r < NH; ++r) l[r] = 0.f;
      float x[NH];
      auto ready = [&](uint32_t i) {  // S of tile i and its values' factors, without waiting
        return __all_sync(0xffffffffu, mbar_test(vfull + 8 * (i & 1u), (i >> 1) & 1u) &&
                                           mbar_test(sfull + 8 * (i & 1u), (i >> 1) & 1u));
      };
      auto load_s = [&](uint32_t i) {
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NH; c += 8) tmem_ld8(tl + (i & 1u) * N + static_cast<uint32_t>(c), x + c);
      };
      bool loaded = false;  // this tile's scores were requested behind the last one's probabilities
#pragma unroll 1
      for (int j = w.j0; j < w.j1; ++j, ++it) {
        const uint32_t buf = it & 1u;
        const int key0 = j >= w.seq.cached ? w.seq.L : ((w.seq.lo >> kBTileLog) + j) * kBTile;
        const int key = key0 + key_in;
        if (!loaded) {
          wait_on(vfull + 8 * buf, (it >> 1) & 1u, abort_flag, a.err);
          wait_on(sfull + 8 * buf, (it >> 1) & 1u, abort_flag, a.err);
          __syncwarp();
          load_s(it);
        }
        const float2 inf = info[(it & 3) * kBTile + key_in];
        const float f = inf.x * qscale;
        const bool there = !(inf.y < 0.f);
        // the values' factor (NaN if it is)
        const float vlog = fmaf(inf.y, 0.f, static_cast<float>(static_cast<int>(__float_as_uint(inf.y) >> 23) - 127));
        const float vinv = pow2_inverse(inf.y) * kBSumUnit;
        const bool own = kTree && j >= w.seq.cached;  // (a tree always has rows of its own)
        const bool masked = own || key0 < all_lo || key0 + kBTile > all_hi || __any_sync(0xffffffffu, !there);
        // of a tree's own rows, bit `lane` of word `quad` of the row's line (there are no more than two words)
        auto tree_seen = [&](int r) {
          const int4 v = *reinterpret_cast<const int4*>(row_tree + (quad & 1) * N + r0 + r);
          const bool in = quad < 2;
          return make_int4(in ? (v.x >> lane) & 1 : 0, in ? (v.y >> lane) & 1 : 0, in ? (v.z >> lane) & 1 : 0,
                           in ? (v.w >> lane) & 1 : 0);
        };
        __syncwarp();
        tmem_ld_wait();
        // scores and values' factors (log2 domain) relative to the rows' references
        auto weigh = [&](float a, float b) {
          return __ffma2_rn(make_float2(a, b), make_float2(f, f), make_float2(vlog, vlog));
        };
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int r = 0; r < NH; r += 4) {
          const float4 t = *reinterpret_cast<const float4*>(row_t + r0 + r);
          const float2 y0 = __fadd2_rn(weigh(x[r], x[r + 1]), make_float2(t.x, t.y));
          const float2 y1 = __fadd2_rn(weigh(x[r + 2], x[r + 3]), make_float2(t.z, t.w));
          x[r] = y0.x; x[r + 1] = y0.y; x[r + 2] = y1.x; x[r + 3] = y1.y;
        }
        if (own) {
#pragma unroll
          for (int r = 0; r < NH; r += 4) {
            const int4 v = tree_seen(r);
            if (v.x == 0) x[r] = -INFINITY;
            if (v.y == 0) x[r + 1] = -INFINITY;
            if (v.z == 0) x[r + 2] = -INFINITY;
            if (v.w == 0) x[r + 3] = -INFINITY;
          }
        } else if (masked) {
#pragma unroll
          for (int r = 0; r < NH; r += 4) {
            const int4 lo = *reinterpret_cast<const int4*>(row_lo + r0 + r), hi = *reinterpret_cast<const int4*>(row_hi + r0 + r);
            if (!there || key < lo.x || key >= hi.x) x[r] = -INFINITY;
            if (!there || key < lo.y || key >= hi.y) x[r + 1] = -INFINITY;
            if (!there || key < lo.z || key >= hi.z) x[r + 2] = -INFINITY;
            if (!there || key < lo.w || key >= hi.w) x[r + 3] = -INFINITY;
          }
        }
#pragma unroll
        for (int r = 0; r < NH; ++r) top[r & 3] = fmaxf(top[r & 3], x[r]);
        top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        if (bar_or(top[0] > kBSlack || *mixed != 0)) {
          // ---- raise the references to the rows' maxima over the tile. Once a tile: a row's weights are then
          // numbers less at least their maximum, and a lift, so that none passes the slack. (The maximum is
          // taken over the same rounded numbers: were the reference subtracted inside the FMA, from 2^27
          // on the largest would pass any slack by its own rounding.)
          __syncwarp();
          load_s(it);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < NH; r += 4) {
            const float4 g = *reinterpret_cast<const float4*>(row_q + r0 + r);
            const float2 g0 = __fmul2_rn(make_float2(x[r], x[r + 1]), make_float2(g.x, g.y));
            const float2 g1 = __fmul2_rn(make_float2(x[r + 2], x[r + 3]), make_float2(g.z, g.w));
            const int4 lo = *reinterpret_cast<const int4*>(row_lo + r0 + r), hi = *reinterpret_cast<const int4*>(row_hi + r0 + r);
            const float2 y0 = weigh(g0.x, g0.y), y1 = weigh(g1.x, g1.y);
            if (own) {
              const int4 v = tree_seen(r);
              x[r] = v.x != 0 ? y0.x : -INFINITY;
              x[r + 1] = v.y != 0 ? y0.y : -INFINITY;
              x[r + 2] = v.z != 0 ? y1.x : -INFINITY;
              x[r + 3] = v.w != 0 ? y1.y : -INFINITY;
              continue;
            }
            x[r] = there && key >= lo.x && key < hi.x ? y0.x : -INFINITY;
            x[r + 1] = there && key >= lo.y && key < hi.y ? y0.y : -INFINITY;
            x[r + 2] = there && key >= lo.z && key < hi.z ? y1.x : -INFINITY;
            x[r + 3] = there && key >= lo.w && key < hi.w ? y1.y : -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < NH; c += 8) {
            const float v = warp_reduce8(x + c, lane, [](float p, float q) { return fmaxf(p, q); });
            if ((lane & 3) == 0) row_red[quad * N + r0 + c + warp_reduce8_row(lane)] = v;
          }
          bar_soft();
          if (threadIdx.x < N) {
            const int r = threadIdx.x;
            const float told = row_t[r];
            const float mx = fmaxf(fmaxf(row_red[r], row_red[N + r]), fmaxf(row_red[2 * N + r], row_red[3 * N + r]));
            const float t = kBLift - mx;
            float shrink = 1.f;
            if (told != kBPadding && mx > -INFINITY && t < told) {
              shrink = told == kBUnseen ? 0.f : ex2_approx(t - told);
              row_t[r] = t;
            }
            row_f[r] = shrink;
          }
          bar_soft();
#pragma unroll
          for (int r = 0; r < NH; r += 4) {
            const float4 g = *reinterpret_cast<const float4*>(row_f + r0 + r);
            l[r] *= g.x; l[r + 1] *= g.y; l[r + 2] *= g.z; l[r + 3] *= g.w;
          }
          if (j > w.j0) {
            wait_on(odone, (it - 1) & 1u, abort_flag, a.err);
            tc_fence_after();
            __syncwarp();
#pragma unroll 1
            for (int c = 0; c < NH; c += 8) {
              float o[8];
              tmem_ld8(tl + static_cast<uint32_t>(2 * N + c), o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] *= row_f[r0 + c + i];
              tmem_st8(tl + static_cast<uint32_t>(2 * N + c), o);
            }
            tmem_st_wait();
            tc_fence_before();
          }
#pragma unroll
          for (int r = 0; r < NH; r += 4) {
            const float4 t = *reinterpret_cast<const float4*>(row_t + r0 + r);
            x[r] += t.x; x[r + 1] += t.y; x[r + 2] += t.z; x[r + 3] += t.w;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty + 8 * buf);
        // ---- probabilities times the values' factors: fp16 operand; without those: fp32 sums
        if (it > 0) wait_on(odone, (it - 1) & 1u, abort_flag, a.err);  // the operand tile is free
#pragma unroll
        for (int c = 0; c < NK; ++c) {
          uint32_t p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * c + 2 * i;
            const float2 e = make_float2(ex2_approx(x[r]), ex2_approx(x[r + 1]));
            const float2 sum = __ffma2_rn(e, make_float2(vinv, vinv), make_float2(l[r], l[r + 1]));
            l[r] = sum.x;
            l[r + 1] = sum.y;
            const __half2 h = __floats2half2_rn(e.x, e.y);
            p[i] = *reinterpret_cast<const uint32_t*>(&h);
          }
          st_shared_v4(to[c], make_uint4(p[0], p[1], p[2], p[3]));
        }
        // the next tile's scores travel while the fence completes (x is free), if they are there
        loaded = j + 1 < w.j1 && ready(it + 1);
        __syncwarp();
        if (loaded) load_s(it + 1);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull);
      }

#pragma unroll
      for (int c = 0; c < NH; c += 8) {
        const float v = warp_reduce8(l + c, lane, [](float p, float q) { return p + q; });
        if ((lane & 3) == 0) row_red[quad * N + r0 + c + warp_reduce8_row(lane)] = v;
      }
      gave = w.j1 < w.seq.tiles;
      if (gave && w.j0 > 0)  // (the range lies inside the item)
        join.leads = BlockParts(range.line, w.start, kSetup, w.seq.tiles).leads(static_cast<int>(blockIdx.x));
      next.next(a);
    }
    auto give = [&]() {  // this range's part is complete
      __threadfence();
      bar_soft();
      if (threadIdx.x == 0) st_release_u64(a.flags + blockIdx.x, a.call);
    };
    if (gave && !join.leads) give();
    if (join.ends || join.leads) {
      block_join<D, NK, kTree>(a, range.line, join, smem, join_full, abort_flag);
      if (join.leads) give();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kBMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Row tiles of equal size, at most 80 rows each (the softmax threads keep a sum and a score of half of
// them in registers).
struct BlockPlan {
  int row_tiles, tile_rows, nk, ctas;
};
BlockPlan block_plan(int B, int G, int Hq, int Hkv, int64_t max_ctx, int sms) {
  BlockPlan p;
  const int rows = G * (Hq / Hkv);
  p.row_tiles = (rows + 79) / 80;
  p.tile_rows = (rows + p.row_tiles - 1) / p.row_tiles;
  p.nk = p.tile_rows <= 16 ? 1 : (p.tile_rows <= 32 ? 2 : (p.tile_rows <= 64 ? 4 : 5));
  const int64_t items = static_cast<int64_t>(B) * Hkv * p.row_tiles;
  // an SM each, as far as there can be tiles
  p.ctas = static_cast<int>(std::min<int64_t>(sms, items * ((max_ctx + kBTile - 1) / kBTile + 1)));
  return p;
}

template <int D, int NK, bool kTree>
int launch_block_t(const BlockArgs& a, const BlockPlan& p, cudaStream_t st) {
  using C = BlockCfg<D, NK>;
  constexpr int kSmem = kTree ? C::kSmemTree : C::kSmem;
  static_assert(kSmem <= 232448, "shared memory");
  static unsigned done = 0;
  auto kern = kv4_attention_kernel<D, NK, kTree>;
  if (!ensure_smem_attr(kern, kSmem, &done)) return fail(DFLASH2_ERR_CUDA, "cudaFuncSetAttribute failed (attention)");
  const cudaError_t e =
      launch_pdl(kern, dim3(static_cast<unsigned>(p.ctas)), dim3(kBThreads), kSmem, st, nullptr, 0, a);
  return e == cudaSuccess ? DFLASH2_OK : fail(DFLASH2_ERR_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
}

template <int D, bool kTree>
int launch_block_d(const BlockArgs& a, const BlockPlan& p, cudaStream_t st) {
  switch (p.nk) {
    case 1: return launch_block_t<D, 1, kTree>(a, p, st);
    case 2: return launch_block_t<D, 2, kTree>(a, p, st);
    case 4: return launch_block_t<D, 4, kTree>(a, p, st);
    default: return launch_block_t<D, 5, kTree>(a, p, st);
  }
}

}  // namespace

size_t kv4_attention_workspace(int B, int G, int Hq, int Hkv, int D, int page_size, int max_pages, int sms) {
  const BlockPlan p = block_plan(B, G, Hq, Hkv, static_cast<int64_t>(max_pages) * page_size, sms);
  const size_t slots = static_cast<size_t>(p.ctas) * 2 * (16 * p.nk);
  return slots * D * sizeof(float) + slots * sizeof(float2) + static_cast<size_t>(p.ctas) * sizeof(unsigned long long);
}

int launch_kv4_attention(const Kv4Attention& r, cudaStream_t st) {
  const BlockPlan p = block_plan(r.B, r.G, r.Hq, r.Hkv, static_cast<int64_t>(r.max_pages) * r.page_size, sm_count());
  BlockArgs a{};
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
  a.tile_rows = p.tile_rows;
  a.row_tiles = p.row_tiles;
  while ((1 << a.page_shift) < r.page_size) ++a.page_shift;
  a.num_pages = r.num_pages;
  a.width = r.max_pages;
  a.cap = r.max_pages * r.page_size;  // (below 2^31: checked)
  a.causal = r.causal;
  a.window = r.window;
  a.scale_log2 = r.scale * 1.4426950408889634f;
  a.out = static_cast<__nv_bfloat16*>(r.out);
  const size_t slots = static_cast<size_t>(p.ctas) * 2 * (16 * p.nk);
  a.part_o = static_cast<float*>(r.workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + slots * r.D);
  a.flags = reinterpret_cast<unsigned long long*>(a.part_ml + slots);
  a.call = next_call_number();
  a.ctas_inverse = ~0ull / static_cast<unsigned long long>(p.ctas);
  a.err = device_error_word();
  if (a.err == nullptr) return fail(DFLASH2_ERR_CUDA, "no device error word");
  if (r.parents != nullptr) return r.D == 64 ? launch_block_d<64, true>(a, p, st) : launch_block_d<128, true>(a, p, st);
  return r.D == 64 ? launch_block_d<64, false>(a, p, st) : launch_block_d<128, false>(a, p, st);
}

}  // namespace dfl
