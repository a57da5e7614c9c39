// A block's rows as a forest: parent indices to the set of each row's ancestors.
#pragma once

#include <cstdint>

namespace dfl {

constexpr int kTreeRows = 64;  // a row's ancestors are the bits of one 64-bit word

// Rows `lane` and `lane + 32` of a tree: bit j of `line` is set if row j is the row itself or one of its
// ancestors; 0: the row is not there.
struct TreeLines {
  uint64_t line[2];
};

// A warp's work. `parent` holds the two rows' parents: an earlier row's index, -1 for a root, less for a row that
// is not there (as rows from `rows` on). A row whose parent is not an earlier row sets `bad` and counts as not
// there, and so does every row below one that is not there. By pointer doubling: after step i a row has taken in
// its 2^i nearest ancestors' bits and points past them, so that six steps reach any root, whatever the depth.
__device__ __forceinline__ TreeLines tree_lines(const int (&parent)[2], int rows, bool& bad) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  TreeLines t;
  int jump[2];
  bad = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = lane + 32 * i;
    const bool there = row < rows && parent[i] >= -1;
    const bool wrong = there && parent[i] >= row;
    bad = bad || wrong;
    t.line[i] = there && !wrong ? 1ull << row : 0ull;
    jump[i] = there && !wrong ? parent[i] : -1;
  }
#pragma unroll 1
  for (int step = 0; step < 6; ++step) {
    uint64_t line[2];
    int next[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t lo = __shfl_sync(0xffffffffu, t.line[0], jump[i] & 31), hi = __shfl_sync(0xffffffffu, t.line[1], jump[i] & 31);
      const int jlo = __shfl_sync(0xffffffffu, jump[0], jump[i] & 31), jhi = __shfl_sync(0xffffffffu, jump[1], jump[i] & 31);
      line[i] = jump[i] >= 32 ? hi : lo;
      next[i] = jump[i] >= 32 ? jhi : jlo;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (jump[i] < 0) continue;
      t.line[i] = line[i] == 0ull ? 0ull : (t.line[i] | line[i]);
      jump[i] = line[i] == 0ull ? -1 : next[i];
    }
  }
  return t;
}

}  // namespace dfl
