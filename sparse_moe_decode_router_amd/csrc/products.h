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
  return grid_launch(units, (a.P + cols - 1) / cols, 4, [&](const Grid& g, unsigned blocks) {
    a.grid = g;
    rows_kernel<S, SEGS, GATED, OUT><<<blocks, S::NT, S::kLds, s>>>(a);
    MOE_HIP(hipGetLastError());
    return (int)MOE_OK;
  });
}

// Gradients of the matrices (grads.hip).
int mats_launch(MatsArgs& a, int type, int out_type, bool al, hipStream_t s);

}  // namespace moe
