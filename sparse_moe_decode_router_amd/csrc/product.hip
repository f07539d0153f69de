// Products of 16-bit rows with 16-bit matrices, y = x W^T (one matrix, or one
// per expert over rows in expert order), and their gradients
//     dx = dy W,   dW = dy^T x
// (the experts' second half beside gated.hip; "How it works" on the Swiftlet
// pages applies k of E experts to each token).  Sums in fp32 on the matrix
// cores; tiles.h has the tiles.
#include "products.h"
#include "stream.h"

namespace moe {
namespace {

// y = x W^T: k and k; dx = dy W: k and p
template <int TYPE, bool PK, int OUT, bool AL> int rows_launch(RowsArgs& a, hipStream_t s) {
  if (few_tiles(a.offsets ? a.E : 0, a.N, a.P)) return rows_grid<Small<TYPE, true, PK, false, AL>, 1, false, OUT>(a, s);
  if constexpr (AL)
    if (wide_rows(a.offsets ? a.E : 0, a.N, a.P)) return rows_grid<Wide<TYPE, true, PK, false>, 1, false, OUT>(a, s);
  return rows_grid<Large<TYPE, true, PK, false, AL>, 1, false, OUT>(a, s);
}
template <int TYPE, int OUT, bool AL> int forward_few(RowsArgs& a, int form, hipStream_t s) {
  // rows of 1024 and more: 8 waves share k.  Shorter ones have not the steps
  // for that: 4 waves, or where blocks are many 2 with 4 tiles each (us, 512 x
  // 2048: 10 rows of 512 experts 9.2, 6.9 and 8.4, 40 rows of 256 26, 23 and 17;
  // 2048 x 512: 10 rows of 512 8.4, 8.5 and 13)
  if (form == 1 && a.K >= 1024) return stream_launch<TYPE, false, 1, 1, 8, 2, OUT, AL>(a, s);
  if (form == 1 && (a.offsets ? max_chunks(a.N, a.E, 16) : 1) * ((a.P + 15) / 16) <= 2048)
    return stream_launch<TYPE, false, 1, 1, 4, 4, OUT, AL>(a, s);
  if (form == 1) return stream_launch<TYPE, false, 4, 1, 2, 2, OUT, AL>(a, s);
  // more columns a block where there are many (32 rows: 4096 -> 4096 14.4 us with
  // 16 columns, 18.9 with 32; 2048 -> 16384 25.6 and 21.4)
  if (a.P <= 8192)
    return form == 2 ? stream_launch<TYPE, false, 1, 2, 4, 4, OUT, AL>(a, s) : stream_launch<TYPE, false, 1, 4, 4, 2, OUT, AL>(a, s);
  return form == 2 ? stream_launch<TYPE, false, 2, 2, 4, 4, OUT, AL>(a, s) : stream_launch<TYPE, false, 2, 4, 4, 2, OUT, AL>(a, s);
}
template <int TYPE, int OUT> int forward_typed(RowsArgs& a, bool al, hipStream_t s) {
  if (const int form = few_rows(a.offsets ? a.E : 0, a.N))
    return al ? forward_few<TYPE, OUT, true>(a, form, s) : forward_few<TYPE, OUT, false>(a, form, s);
  return al ? rows_launch<TYPE, true, OUT, true>(a, s) : rows_launch<TYPE, true, OUT, false>(a, s);
}
template <int TYPE> int dx_typed(RowsArgs& a, bool al, hipStream_t s) {
  return al ? rows_launch<TYPE, false, TYPE, true>(a, s) : rows_launch<TYPE, false, TYPE, false>(a, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_linear(const void* w, size_t w_stride, int32_t E, const void* x, int32_t type, int32_t N,
                          int32_t n_in, int32_t n_out, const int32_t* offsets, void* y, int32_t y_type,
                          hipStream_t s) {
  MOE_TRY(product_check(E, type, N, n_in, n_out, offsets));
  MOE_CHECK((y_type == type || y_type == MOE_TYPE_F32) && matrices_ok(w, w_stride, E, (long)n_in * n_out));
  if (N == 0) return MOE_OK;
  MOE_CHECK(w && x && y && aligned(x, 2) && aligned(y, type_size(y_type)));
  RowsArgs a{};
  a.q = static_cast<const uint8_t*>(x);
  a.q_ld = a.p_ld = a.K = n_in;
  a.p = static_cast<const uint8_t*>(w);
  a.p_stride = w_stride;
  a.P = n_out;
  a.offsets = offsets;
  a.E = E;
  a.N = N;
  a.out = y;
  const bool al = whole_pieces({n_in, n_out}, {w, x, y}, {w_stride});
  if (type == MOE_TYPE_BF16)
    return y_type == type ? forward_typed<MOE_TYPE_BF16, MOE_TYPE_BF16>(a, al, s)
                          : forward_typed<MOE_TYPE_BF16, MOE_TYPE_F32>(a, al, s);
  return y_type == type ? forward_typed<MOE_TYPE_F16, MOE_TYPE_F16>(a, al, s)
                        : forward_typed<MOE_TYPE_F16, MOE_TYPE_F32>(a, al, s);
}

extern "C" int moe_linear_backward(const void* dy, const void* w, size_t w_stride, int32_t E, const void* x,
                                   int32_t type, int32_t N, int32_t n_in, int32_t n_out, const int32_t* offsets,
                                   void* dx, void* dw, size_t dw_stride, int32_t dw_type, hipStream_t s) {
  MOE_TRY(product_check(E, type, N, n_in, n_out, offsets));
  MOE_CHECK(dx || dw);
  MOE_CHECK(!dx || matrices_ok(w, w_stride, E, (long)n_in * n_out));
  MOE_CHECK(!dw || ((dw_type == type || dw_type == MOE_TYPE_F32) &&
                    matrices_ok(dw, dw_stride, E, (long)n_in * n_out, type_size(dw_type))));
  MOE_CHECK(N == 0 || (dy && aligned(dy, 2) && (!dx || (w && aligned(dx, 2))) && (!dw || (x && aligned(x, 2)))));
  if (dx && N > 0) {
    RowsArgs a{};
    a.q = static_cast<const uint8_t*>(dy);
    a.q_ld = a.K = n_out;
    a.p = static_cast<const uint8_t*>(w);
    a.p_stride = w_stride;
    a.p_ld = a.P = n_in;
    a.offsets = offsets;
    a.E = E;
    a.N = N;
    a.out = dx;
    const bool al = whole_pieces({n_in, n_out}, {w, dy, dx}, {w_stride});
    MOE_TRY(type == MOE_TYPE_BF16 ? dx_typed<MOE_TYPE_BF16>(a, al, s) : dx_typed<MOE_TYPE_F16>(a, al, s));
  }
  if (!dw) return MOE_OK;
  MatsArgs m{};
  m.q = static_cast<const uint8_t*>(dy);
  m.p = static_cast<const uint8_t*>(x);
  m.q_ld = m.Q = n_out;
  m.p_ld = m.P = n_in;
  m.mats = 1;
  m.offsets = offsets;
  m.E = E;
  m.N = N;
  m.out = dw;
  m.out_stride = dw_stride;
  return mats_launch(m, type, dw_type, whole_pieces({n_in, n_out}, {dy, x, dw}, {dw_stride}), s);
}
