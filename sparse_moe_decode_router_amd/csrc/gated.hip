// The gated block of an expert's feed-forward network, in 16-bit types and with
// its gradients, for rows of one matrix pair or rows in expert order:
//     g = x Wg^T, u = x Wu^T, h = act(g) u
//     dg = dh u act'(g), du = dh act(g)
//     dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
// (SwiGLU of the routed experts, layer.py's reading of the Swiftlet pages, and
// its relatives).  Both products and the activation are one kernel: a wave
// holds the same 32 columns of g and of u in the same registers, so h is formed
// on the fp32 sums and rounded once.  For the gradients g and u are saved in
// fp32: dg and du have to be rounded to the rows' type, as operands of the
// matrix cores, which alone moves dx and dW by as much as their own rounding
// does (in all sqrt 2 of a rounding in norm, 1.35 to 1.45 measured; of a few
// hundred elements 1.3 to 1.6); g and u rounded as well moved them by 1.8.  Kept whole they
// would be two operands each, with twice the products of the backward pass.
// In fp16 it also has fp16's range (the header says what becomes of dg and du
// outside it): a scale would have to be one a row for dx and one a column of an
// expert for dW, from a pass over dh and pre of its own.
#include "products.h"
#include "stream.h"

namespace moe {
namespace {

template <int TYPE, bool AL> int forward(RowsArgs& a, hipStream_t s) {
  const int form = few_rows(a.offsets ? a.E : 0, a.N);
  if (form == 1)                                // as product.hip
    return a.K >= 1024 ? stream_launch<TYPE, true, 2, 1, 8, 4, TYPE, AL>(a, s) : stream_launch<TYPE, true, 2, 1, 4, 4, TYPE, AL>(a, s);
  if (form == 2) return stream_launch<TYPE, true, 2, 2, 4, 2, TYPE, AL>(a, s);
  if (form == 4) return stream_launch<TYPE, true, 2, 4, 4, 1, TYPE, AL>(a, s);
  if (few_tiles(a.offsets ? a.E : 0, a.N, 2l * a.P)) return rows_grid<Small<TYPE, true, true, true, AL>, 1, true, TYPE>(a, s);
  if constexpr (AL)
    if (wide_rows(a.offsets ? a.E : 0, a.N, 2l * a.P)) return rows_grid<Wide<TYPE, true, true, true>, 1, true, TYPE>(a, s);
  return rows_grid<Large<TYPE, true, true, true, AL>, 1, true, TYPE>(a, s);
}
template <int TYPE, bool AL> int backward_dx(RowsArgs& a, hipStream_t s) {
  if (few_tiles(a.offsets ? a.E : 0, a.N, a.P)) return rows_grid<Small<TYPE, true, false, false, AL>, 2, false, TYPE>(a, s);
  if constexpr (AL)
    if (wide_rows(a.offsets ? a.E : 0, a.N, a.P)) return rows_grid<Wide<TYPE, true, false, false>, 2, false, TYPE>(a, s);
  return rows_grid<Large<TYPE, true, false, false, AL>, 2, false, TYPE>(a, s);
}

// VN consecutive fp32 values
template <int VN> __device__ __forceinline__ void load_f32(const float* p, float (&v)[VN]) {
  constexpr int kN = VN == 8 ? 4 : 1;
#pragma unroll
  for (int h = 0; h < VN / kN; ++h) {
    const Vec<MOE_TYPE_F32, kN> e = vec_load<MOE_TYPE_F32, kN>(p + h * kN);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[h * kN + i] = e.e[i];
  }
}
// dg | du [N][2 I] from dh [N][I] and pre = g | u [N][2 I], VN elements a
// thread: bound by HBM (4096 x 8192: 73 us, 6.4 TB/s).
template <int TYPE, int VN>
__global__ __launch_bounds__(256) void slope_kernel(const typename El<TYPE>::raw* dh, const float* pre,
                                                    typename El<TYPE>::raw* out, int I, long pieces, int act) {
  const int row_pieces = I / VN;
  const long first = (long)blockIdx.x * 256;
  const long row0 = first / row_pieces;
  const unsigned in = (unsigned)(first - row0 * row_pieces) + threadIdx.x;
  if (first + threadIdx.x >= pieces) return;
  const long row = row0 + in / (unsigned)row_pieces;
  const int c = (int)(in % (unsigned)row_pieces) * VN;
  const Vec<TYPE, VN> d = vec_load<TYPE, VN>(dh + row * I + c);
  float g[VN], u[VN];
  load_f32<VN>(pre + 2 * row * I + c, g);
  load_f32<VN>(pre + (2 * row + 1) * I + c, u);
  Vec<TYPE, VN> dg, du;
#pragma unroll
  for (int i = 0; i < VN; ++i) {
    float f;
    const float df = act_slope(act, g[i], &f), v = El<TYPE>::up(d.e[i]);
    dg.e[i] = El<TYPE>::down(v * u[i] * df);
    du.e[i] = El<TYPE>::down(v * f);
  }
  vec_store<TYPE, VN>(out + 2 * row * I + c, dg);
  vec_store<TYPE, VN>(out + (2 * row + 1) * I + c, du);
}
template <int TYPE>
int slope(const void* dh, const float* pre, void* out, long N, int I, int act, hipStream_t s) {
  typedef typename El<TYPE>::raw raw;
  const int vn = I % 8 == 0 ? 8 : 1;
  const long per = (1l << 30) / (I / vn);       // rows a launch
  for (long r = 0; r < N; r += per) {
    const long rows = N - r < per ? N - r : per, pieces = rows * (I / vn);
    const raw* d = static_cast<const raw*>(dh) + r * I;
    const float* p = pre + 2 * r * I;
    raw* o = static_cast<raw*>(out) + 2 * r * I;
    const unsigned blocks = (unsigned)((pieces + 255) / 256);
    if (vn == 8)
      slope_kernel<TYPE, 8><<<blocks, 256, 0, s>>>(d, p, o, I, pieces, act);
    else
      slope_kernel<TYPE, 1><<<blocks, 256, 0, s>>>(d, p, o, I, pieces, act);
    MOE_HIP(hipGetLastError());
  }
  return MOE_OK;
}

bool act_ok(int act) { return act == MOE_ACT_SILU || act == MOE_ACT_GELU || act == MOE_ACT_GELU_TANH; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_gated(const void* w_gate, size_t gate_stride, const void* w_up, size_t up_stride, int32_t E,
                         const void* x, int32_t type, int32_t N, int32_t d, int32_t I, const int32_t* offsets,
                         int32_t act, void* h, float* pre, hipStream_t s) {
  MOE_TRY(product_check(E, type, N, d, I, offsets));
  MOE_CHECK(act_ok(act) && matrices_ok(w_gate, gate_stride, E, (long)d * I) &&
            matrices_ok(w_up, up_stride, E, (long)d * I));
  if (N == 0) return MOE_OK;
  MOE_CHECK(w_gate && w_up && x && h && aligned(x, 2) && aligned(h, 2) && aligned(pre, 4));
  RowsArgs a{};
  a.q = static_cast<const uint8_t*>(x);
  a.q_ld = a.p_ld = a.K = d;
  a.p = static_cast<const uint8_t*>(w_gate);
  a.p2 = static_cast<const uint8_t*>(w_up);
  a.p_stride = gate_stride;
  a.p2_stride = up_stride;
  a.P = I;
  a.offsets = offsets;
  a.E = E;
  a.N = N;
  a.act = act;
  a.out = h;
  a.pre = pre;
  if (whole_pieces({d, I}, {w_gate, w_up, x, h, pre}, {gate_stride, up_stride}))
    return type == MOE_TYPE_BF16 ? forward<MOE_TYPE_BF16, true>(a, s) : forward<MOE_TYPE_F16, true>(a, s);
  return type == MOE_TYPE_BF16 ? forward<MOE_TYPE_BF16, false>(a, s) : forward<MOE_TYPE_F16, false>(a, s);
}

extern "C" size_t moe_gated_backward_workspace_bytes(int32_t N, int32_t I) {
  return N < 0 || N > (1 << 30) || I < 1 || I > kMostSize ? 0 : (size_t)N * I * 4 + 256;
}

extern "C" int moe_gated_backward(const void* dh, const float* pre, const void* w_gate, size_t gate_stride,
                                  const void* w_up, size_t up_stride, int32_t E, const void* x, int32_t type,
                                  int32_t N, int32_t d, int32_t I, const int32_t* offsets, int32_t act, void* dx,
                                  void* dw_gate, size_t dw_gate_stride, void* dw_up, size_t dw_up_stride,
                                  int32_t dw_type, void* ws, size_t ws_bytes, hipStream_t s) {
  MOE_TRY(product_check(E, type, N, d, I, offsets));
  MOE_CHECK(act_ok(act) && (dx || dw_gate) && !dw_gate == !dw_up);
  MOE_CHECK(!dx || (matrices_ok(w_gate, gate_stride, E, (long)d * I) && matrices_ok(w_up, up_stride, E, (long)d * I)));
  MOE_CHECK(!dw_gate || ((dw_type == type || dw_type == MOE_TYPE_F32) &&
                         matrices_ok(dw_gate, dw_gate_stride, E, (long)d * I, type_size(dw_type)) &&
                         matrices_ok(dw_up, dw_up_stride, E, (long)d * I, type_size(dw_type))));
  MOE_CHECK(N == 0 || (dh && pre && ws && aligned(dh, 2) && aligned(pre, 4) && aligned(ws, 16) &&
                       ws_bytes >= moe_gated_backward_workspace_bytes(N, I) &&
                       (!dx || (w_gate && w_up && aligned(dx, 2))) && (!dw_gate || (x && aligned(x, 2)))));
  if (N > 0) {
    MOE_TRY(type == MOE_TYPE_BF16 ? slope<MOE_TYPE_BF16>(dh, pre, ws, N, I, act, s)
                                  : slope<MOE_TYPE_F16>(dh, pre, ws, N, I, act, s));
    if (dx) {
      RowsArgs a{};
      a.q = static_cast<const uint8_t*>(ws);
      a.q_ld = 2l * I;
      a.K = I;
      a.p = static_cast<const uint8_t*>(w_gate);
      a.p2 = static_cast<const uint8_t*>(w_up);
      a.p_stride = gate_stride;
      a.p2_stride = up_stride;
      a.p_ld = a.P = d;
      a.offsets = offsets;
      a.E = E;
      a.N = N;
      a.out = dx;
      const bool al = whole_pieces({d, I}, {w_gate, w_up, ws, dx}, {gate_stride, up_stride});
      MOE_TRY(type == MOE_TYPE_BF16
                  ? (al ? backward_dx<MOE_TYPE_BF16, true>(a, s) : backward_dx<MOE_TYPE_BF16, false>(a, s))
                  : (al ? backward_dx<MOE_TYPE_F16, true>(a, s) : backward_dx<MOE_TYPE_F16, false>(a, s)));
    }
  }
  if (!dw_gate) return MOE_OK;
  MatsArgs m{};
  m.q = static_cast<const uint8_t*>(ws);
  m.p = static_cast<const uint8_t*>(x);
  m.q_ld = 2l * I;
  m.Q = I;
  m.p_ld = m.P = d;
  m.mats = 2;
  m.offsets = offsets;
  m.E = E;
  m.N = N;
  m.out = dw_gate;
  m.out2 = dw_up;
  m.out_stride = dw_gate_stride;
  m.out2_stride = dw_up_stride;
  return mats_launch(m, type, dw_type, whole_pieces({d, I}, {ws, x, dw_gate, dw_up}, {dw_gate_stride, dw_up_stride}), s);
}
