// Sorted rows cut into chunks that do not cross an expert's border, numbered in
// expert order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct RowChunk {
  int e;        // expert, -1 past the last chunk
  int start;    // first row
  int n;        // rows (0..size)
  int index;    // of the chunk within its expert
  int of;       // chunks of that expert
  int multi;    // chunks of earlier experts that have more than one
};
struct ChunkTotals {
  int chunks, multi;
};

// Chunk j of `size` rows of the buckets offsets[0..E] (E <= 1024).  EMPTY: an
// expert without rows has one chunk of none.  Every wave finds its own: lane l
// holds experts l*per .., the chunks before them come from a wave scan.
// Offsets that do not describe N rows give no row outside them.
template <bool EMPTY>
__device__ __forceinline__ RowChunk find_chunk(const int32_t* __restrict__ offsets, int E, long N, long j, int size,
                                               ChunkTotals* totals) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;                // <= 16
  int off[17];
#pragma unroll
  for (int u = 0; u <= 16; ++u) {
    off[u] = 0;
    if (u <= per) {
      const int e = lane * per + u;
      off[u] = offsets[e < E ? e : E];
    }
  }
  auto chunks_of = [&](int u) {
    const int rows = off[u + 1] - off[u];
    const bool real = u < per && lane * per + u < E;
    return !real ? 0 : rows > 0 ? (rows + size - 1) / size : EMPTY ? 1 : 0;
  };
  int mine = 0, mm = 0;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int c = chunks_of(u);
    mine += c;
    mm += c > 1 ? c : 0;
  }
  int incl = mine, mincl = mm;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int v = __shfl_up(incl, s, 64), v2 = __shfl_up(mincl, s, 64);
    if (lane >= s) {
      incl += v;
      mincl += v2;
    }
  }
  if (totals) *totals = ChunkTotals{__builtin_amdgcn_readlane(incl, 63), __builtin_amdgcn_readlane(mincl, 63)};
  RowChunk r{-1, 0, 0, 0, 0, 0};
  const uint64_t past = __ballot((long)incl > j);
  if (past == 0) return r;
  const int owner = __ffsll((unsigned long long)past) - 1;
  int left = (int)j - (incl - mine), multi = mincl - mm;
  bool found = false;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int c = chunks_of(u);
    if (!found && left < c) {
      const int rows = off[u + 1] - off[u] - left * size;
      r = RowChunk{lane * per + u, off[u] + left * size, rows < size ? rows : size, left, c, multi};
      found = true;
    }
    left -= c;
    multi += c > 1 ? c : 0;
  }
  r.e = __builtin_amdgcn_readlane(r.e, owner);
  r.start = __builtin_amdgcn_readlane(r.start, owner);
  r.n = __builtin_amdgcn_readlane(r.n, owner);
  r.index = __builtin_amdgcn_readlane(r.index, owner);
  r.of = __builtin_amdgcn_readlane(r.of, owner);
  r.multi = __builtin_amdgcn_readlane(r.multi, owner);
  if (r.start < 0 || (long)r.start >= N || r.n < 0) r.start = r.n = 0;
  if ((long)r.start + r.n > N) r.n = (int)(N - r.start);
  return r;
}

// The most chunks that N rows in E buckets can make.
inline long max_chunks(long N, int E, int size, bool empty) {
  const long ne = N < E ? N : E;                // each bucket with rows makes at most one short chunk
  return ne + (N - ne) / size + (empty ? E - ne : 0);
}

}  // namespace moe
