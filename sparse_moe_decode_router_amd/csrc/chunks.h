// Chunks of the rows that moe_sort_tokens brings into expert order.
#pragma once

#include "device.h"

namespace moe {

// Sorted rows are cut into chunks of `size` that do not cross an expert's
// border, numbered in expert order.
struct RowChunk {
  bool any;     // false past the last chunk
  int slot;     // of its expert
  int start;    // first row
  int n;        // rows (0..size)
};

// A border outside 0 .. N is taken as the nearer of the two, wherever borders
// are read.
__device__ __forceinline__ int row_border(int at, int N) { return min(max(at, 0), N); }

// Chunk j.  Every wave finds its own: borders and slots of all experts in
// coalesced loads, all in flight at once (lane l holds experts l, l + 64, ..),
// chunks counted by wave scans of 64 experts.  Where borders fall, the chunk's
// rows are some within N.
__device__ __forceinline__ RowChunk find_chunk(const int32_t* __restrict__ offsets,
                                               const int32_t* __restrict__ slot_table, int E, long N, long j,
                                               int size) {
  constexpr int kU = 16;                        // E <= 1024
  const int lane = threadIdx.x & 63;
  int off[kU + 1], slots[kU];
#pragma unroll
  for (int u = 0; u <= kU; ++u) {
    off[u] = 0;
    if (u < kU) slots[u] = 64 * u + lane;
    if (64 * u <= E) {
      const int e = 64 * u + lane;
      off[u] = offsets[e < E ? e : E];
      if (u < kU && slot_table) slots[u] = slot_table[e < E ? e : E - 1];
    }
  }
  RowChunk r{false, 0, 0, 0};
  int before = 0;                               // chunks of the experts of earlier u
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    if (64 * u < E && !r.any) {
      // the next lane's border (lane 63: the first of the next 64)
      const int next = __builtin_amdgcn_update_dpp(__builtin_amdgcn_readlane(off[u + 1], 0), off[u], 0x130, 0xF, 0xF, false);
      // (not where they are loaded: each load would be waited for before the next, 9.2 us
      // in place of 6.8 for ten rows of 512 experts, 512 -> 2048)
      const int first = row_border(off[u], (int)N), end = row_border(next, (int)N);
      const int rows = 64 * u + 63 < E || lane < E - 64 * u ? end - first : 0;
      const int c = rows > 0 ? (int)((unsigned)(rows + size - 1) / (unsigned)size) : 0;
      const int incl = wave_scan(c) + before;
      const uint64_t past = __ballot((long)incl > j);
      if (past != 0) {
        const int owner = __ffsll((unsigned long long)past) - 1;
        const int skip = ((int)j - __builtin_amdgcn_readlane(incl - c, owner)) * size;
        const int left = __builtin_amdgcn_readlane(rows, owner) - skip;
        r = RowChunk{true, __builtin_amdgcn_readlane(slots[u], owner), __builtin_amdgcn_readlane(first, owner) + skip,
                     left < size ? left : size};
      }
      before = __builtin_amdgcn_readlane(incl, 63);
    }
  }
  if (r.start < 0 || (long)r.start >= N || r.n < 0) r.start = r.n = 0;
  if ((long)r.start + r.n > N) r.n = (int)(N - r.start);
  return r;
}

// The most chunks that N rows in E buckets can make.
inline long max_chunks(long N, int E, int size) {
  const long ne = N < E ? N : E;                // each bucket with rows makes at most one short chunk
  return ne + (N - ne) / size;
}

}  // namespace moe
