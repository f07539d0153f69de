// Checks and launches that the 16-bit products share (product.hip, gated.hip).
#pragma once

#include <initializer_list>

#include "tiles.h"

namespace moe {

constexpr int kMostSize = 1 << 20;              // of a row, so that a tile's offsets fit 31 bits

// Sizes, type and borders of a product of N rows of n_in with E matrices.
inline int product_check(int E, int type, long N, long n_in, long n_out, const int32_t* offsets) {
  MOE_CHECK((type == MOE_TYPE_BF16 || type == MOE_TYPE_F16) && N >= 0 && n_in >= 1 && n_out >= 1 && E >= 1 &&
            E <= 1024 && (offsets || E == 1) && aligned(offsets, 4));
  return n_in > kMostSize || n_out > kMostSize || N > (1 << 30) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
inline bool matrices_ok(const void* w, size_t stride, int E, long elements, int size = 2) {
  return aligned(w, size) && stride % size == 0 && (E == 1 || stride >= (size_t)elements * size);
}
// Rows are whole 16-byte pieces at 16-byte addresses.
inline bool whole_pieces(std::initializer_list<int> sizes, std::initializer_list<const void*> at,
                         std::initializer_list<size_t> strides) {
  bool ok = true;
  for (int v : sizes) ok = ok && v % 8 == 0;
  for (const void* p : at) ok = ok && aligned(p, 16);
  for (size_t v : strides) ok = ok && v % 16 == 0;
  return ok;
}

template <class S, int SEGS, bool GATED, int OUT> int rows_grid(RowsArgs& a, hipStream_t s) {
  const long units = a.offsets ? max_chunks(a.N, a.E, S::BQ) : (a.N + S::BQ - 1) / S::BQ;
  const int cols = GATED ? S::BP / 2 : S::BP;
  // (experts: 2 chunks a group, 1 to 3 % better than 4)
  return grid_launch(units, (a.P + cols - 1) / cols, a.offsets ? 2 : 4, [&](const Grid& g, unsigned blocks) {
    a.grid = g;
    rows_kernel<S, SEGS, GATED, OUT><<<blocks, S::NT, kBlockLds<S, OUT>, s>>>(a);
    MOE_HIP(hipGetLastError());
    return (int)MOE_OK;
  });
}

// The form of a product of N rows, in E buckets or (E 0) of one matrix: 0 tiles
// through LDS, or NT (1, 2, 4): 16 NT rows a block of stream.h.
// One matrix: up to 64 rows (us, streamed and in tiles: 16 x 4096 -> 4096 11 and
// 21, 64 21.4 and 22.2, 64 x 2048 -> 16384 28 and 42).  Experts: up to 8 rows a
// bucket; more of them fill a second chunk, for which W is read again (2048 ->
// 2 x 512 of 512, 5 rows 407 and 454, 10 rows 467 and 459; 2048 -> 2048 of 64, 8
// rows 115 and 135, 16 rows 172 and 135).  The borders are on the device, so this
// goes by the average bucket: rows that are all one expert's are streamed too, and
// its matrix read for each 16 of them (4096 rows of 512 experts, 2048 -> 512: 264 us
// evenly, 182 in one bucket, 17 as one matrix's).
inline int few_rows(int E, long N) {
  if (E) return N <= 8l * E ? 1 : 0;
  return N > 64 ? 0 : N > 32 ? 4 : N > 16 ? 2 : 1;
}

// Whether tiles of 128 x 128 would be few for the 256 CUs, so that 64 x 64 are
// better (us, small and large: 4096 -> 4096 of 512 rows 35 and 53, of 1024 rows,
// 256 tiles, 61 and 54).
inline bool few_tiles(int E, long N, long P) {
  const long chunks = E ? (N < E ? N : E * ((N / E + 127) / 128)) : (N + 127) / 128;
  return chunks * ((P + 127) / 128) <= 128;
}
// Whether tiles of 256 x 256 (one a CU, 1.12 times the rate) take less than
// those of 128 x 128 (`slots` a CU) for `units` matrices of q x p, in whole rounds of the 256 CUs.
// Measured (16-bit, wide against large): 4096 x 4096 -> 4096 115 and 127 us, 4160
// x 4160 -> 4160 194 and 172, 4096 x 8192 -> 2048 564 and 382.
inline bool wide_better(long units, long q, long p, int slots) {
  const long wide = units * ((q + 255) / 256) * ((p + 255) / 256);
  const long large = units * ((q + 127) / 128) * ((p + 127) / 128);
  return (wide + 255) / 256 * 4 < 1.12 * ((large + 256 * slots - 1) / (256 * slots) * slots);
}
// The same for rows: buckets of 512 rows and more, which fill the taller tile.
inline bool wide_rows(int E, long N, long P) {
  const long rows = E ? N / E : N;
  return rows >= 512 && wide_better(E ? E : 1, rows, P, 2);
}

// Gradients of the matrices (grads.hip).
int mats_launch(MatsArgs& a, int type, int out_type, bool al, hipStream_t s);

}  // namespace moe
