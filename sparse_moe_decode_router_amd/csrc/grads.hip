// Gradients of the experts' matrices: dW[q][p] = sum over an expert's rows of
// dy[row][q] x[row][p] (product.hip, gated.hip), an expert without rows zeros.
// Both operands lie with k (the rows) apart: tiles.h reads them turned.
#include "products.h"

namespace moe {
namespace {

template <class S, int OUT> int launch(MatsArgs& a, hipStream_t s) {
  a.q_tiles = (a.Q + S::BQ - 1) / S::BQ;
  return grid_launch((long)a.E * a.mats * a.q_tiles, (a.P + S::BP - 1) / S::BP, 4, [&](const Grid& g, unsigned blocks) {
    a.grid = g;
    mats_kernel<S, OUT><<<blocks, S::NT, kBlockLds<S, OUT>, s>>>(a);
    MOE_HIP(hipGetLastError());
    return (int)MOE_OK;
  });
}
template <int TYPE, int OUT, bool AL> int sized(MatsArgs& a, hipStream_t s) {
  // (us, small and larger tiles: 1024 x 1024 of 1024 rows 10.4 and 17, 2048 x 2048
  // of 256 rows, 256 tiles, 11.1 and 7.8; 128 x 128 and 256 x 256: 256 experts of
  // 128 rows, 2 x 512 x 2048 388 and 374, 512 x 2048 184 and 175, 4096 rows, 2 x 8192
  // x 2048 284 and 262, 16 experts of 1024 rows, 1024 x 1024 40 and 37)
  const long tiles = (long)a.E * a.mats * ((a.Q + 127) / 128) * ((a.P + 127) / 128);
  if (tiles <= 128) return launch<Small<TYPE, false, false, false, AL>, OUT>(a, s);
  if constexpr (AL)
    if (wide_better((long)a.E * a.mats, a.Q, a.P, 3)) return launch<Wide<TYPE, false, false, false>, OUT>(a, s);
  return launch<Mats<TYPE, AL>, OUT>(a, s);
}
template <int TYPE> int typed(MatsArgs& a, int out_type, bool al, hipStream_t s) {
  if (out_type == MOE_TYPE_F32) return al ? sized<TYPE, MOE_TYPE_F32, true>(a, s) : sized<TYPE, MOE_TYPE_F32, false>(a, s);
  return al ? sized<TYPE, TYPE, true>(a, s) : sized<TYPE, TYPE, false>(a, s);
}

}  // namespace

int mats_launch(MatsArgs& a, int type, int out_type, bool al, hipStream_t s) {
  return type == MOE_TYPE_BF16 ? typed<MOE_TYPE_BF16>(a, out_type, al, s) : typed<MOE_TYPE_F16>(a, out_type, al, s);
}

}  // namespace moe
