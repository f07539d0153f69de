// Products in 8-bit floating point (e4m3) with a scale for every 128 inputs of
// a row of x and every 128 x 128 block of W, and the quantisation of both.
//
//     code = e4m3(448 v / a), scale = a / 448, a the block's largest |v|
//     y[p][o] = sum_b sx[p][b] sw[o / 128][b] sum_{j in b} x[p][j] w[o][j]
//
// 448 v is exact for 16-bit v and the quotient is rounded once before it is
// rounded to the code, so codes are those of exact arithmetic, ties included.
// A block's sum of 128 products runs on v_mfma_f32_32x32x64_f8f6f4 (no scales
// of its own), from zero, and is then added with its scales to the running fp32
// sum.  The instruction adds the products of 8 consecutive inputs at once and
// drops of each what is below 2^-13 of the largest's power of two (measured;
// about 1e-5 of a random product, the codes' own rounding is 2^-4); its sums of
// these are fp32.  It has twice the rate of the 16-bit products.
#include "products.h"
#include "stream.h"

namespace moe {
namespace {

constexpr int kBlock = 128;
constexpr float kMax = 448.f, kSmallest = 0x1p-96f, kLarge = 0x1p64f;
constexpr int kNormal = 0x108;                  // v_cmp_class: normal numbers of either sign
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ------------------------------------------------------------ quantisation
// A block with the largest magnitude `top`: codes are e4m3((v m) / a), m 448 or
// (so that 448 v stays finite) 448 2^-32 with a smaller by as much.
struct Block {
  float a, inv, m, scale;
};
__device__ __forceinline__ Block block_of(float top) {
  Block b;
  top = top < kSmallest ? kSmallest : top;
  b.scale = top / kMax;
  const float down = top > kLarge ? 0x1p-32f : 1.f;
  b.m = kMax * down;
  b.a = top * down;
  b.inv = __builtin_amdgcn_rcpf(b.a);
  return b;
}
// The quotient, rounded once: an estimate and its exact remainder (a quotient
// that is a code or a border between two comes out as it is).  The division
// itself, with its care for extremes that cannot occur, made the kernel bound
// by its instructions (32768 x 2048: 58 us).
__device__ __forceinline__ float quotient(const Block& b, float v) {
  const float t = v * b.m, q = t * b.inv;
  return __builtin_copysignf(fmaf(fmaf(-q, b.a, t), b.inv, q), v);
}

// A thread's 8 elements of a row: consecutive ones (VN 8), or every `step`th;
// zeros past `have`.
template <int TYPE, int VN>
__device__ __forceinline__ void load8(const typename El<TYPE>::raw* p, int step, int have, float (&v)[8]) {
  if constexpr (VN == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (have >= 8) {
      constexpr int kN = El<TYPE>::kN;
#pragma unroll
      for (int h = 0; h < 8 / kN; ++h) {
        const Vec<TYPE, kN> e = vec_load<TYPE, kN>(p + h * kN);
#pragma unroll
        for (int i = 0; i < kN; ++i) v[h * kN + i] = El<TYPE>::up(e.e[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i * step < have ? El<TYPE>::up(p[i * step]) : 0.f;
  }
}
template <int VN> __device__ __forceinline__ void store8(uint8_t* p, int step, int have, const Block& b, const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(b, v[4 * h]), quotient(b, v[4 * h + 1]), 0, false);
    w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quotient(b, v[4 * h + 2]), quotient(b, v[4 * h + 3]), c, true);
  }
  if constexpr (VN == 8) {
    if (have >= 8) *reinterpret_cast<uint64_t*>(p) = w[0] | (uint64_t)w[1] << 32;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * step < have) p[i * step] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
  }
}
__device__ __forceinline__ float max16(float v) {               // over each 16 lanes
#pragma unroll
  for (int s = 1; s < 16; s *= 2) v = fmaxf(v, __shfl_xor(v, s, 64));
  return v;
}

// Rows: 16 lanes a block of 128 inputs.
template <int TYPE, int VN>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const typename El<TYPE>::raw* x, int n, int blocks,
                                                            long total, uint8_t* codes, float* scales) {
  const long first = (long)blockIdx.x * 16;
  const long row0 = first / blocks;
  const unsigned in = (unsigned)(first - row0 * blocks) + threadIdx.x / 16;
  if (first + threadIdx.x / 16 >= total) return;
  const long row = row0 + in / (unsigned)blocks;
  const int b = (int)(in % (unsigned)blocks), j = threadIdx.x & 15;
  const int c = b * kBlock + (VN == 8 ? 8 * j : j);
  const int end = n < (b + 1) * kBlock ? n : (b + 1) * kBlock;
  float v[8];
  load8<TYPE, VN>(x + row * n + c, 16, end - c, v);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
  const Block q = block_of(max16(top));
  store8<VN>(codes + row * n + c, 16, end - c, q, v);
  if (j == 0) scales[row * blocks + b] = q.scale;
}

// 128 x 128: a block of threads each, 16 lanes a row, 8 turns of 16 rows.
template <int TYPE, int VN>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const typename El<TYPE>::raw* x, int rows, int n,
                                                              int row_blocks, int blocks, long block0, uint8_t* codes,
                                                              float* scales) {
  __shared__ float tops[4];
  const long id = block0 + blockIdx.x;
  const long m = id / ((long)row_blocks * blocks);
  const int in = (int)(id - m * ((long)row_blocks * blocks));
  const int rb = in / blocks, b = in - rb * blocks, j = threadIdx.x & 15;
  const int c = b * kBlock + (VN == 8 ? 8 * j : j);
  const int end = n < (b + 1) * kBlock ? n : (b + 1) * kBlock;
  float v[8][8];
  float top = 0.f;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const int row = rb * kBlock + 16 * t + threadIdx.x / 16;
    load8<TYPE, VN>(x + (m * rows + row) * n + c, 16, row < rows ? end - c : 0, v[t]);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[t][i]));
  }
  top = max16(top);
  top = fmaxf(top, __shfl_xor(top, 16, 64));
  top = fmaxf(top, __shfl_xor(top, 32, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  const Block q = block_of(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const int row = rb * kBlock + 16 * t + threadIdx.x / 16;
    store8<VN>(codes + (m * rows + row) * n + c, 16, row < rows ? end - c : 0, q, v[t]);
  }
  if (threadIdx.x == 0) scales[id] = q.scale;
}

template <int TYPE, int VN>
int quantize(const void* xv, long count, int rows, int n, int block_rows, uint8_t* codes, float* scales, hipStream_t s) {
  typedef typename El<TYPE>::raw raw;
  const raw* x = static_cast<const raw*>(xv);
  const int blocks = (n + kBlock - 1) / kBlock;
  if (block_rows == 1) {
    const long all = count * rows, per = (1l << 26) / blocks;   // rows a launch
    for (long r = 0; r < all; r += per) {
      const long total = (all - r < per ? all - r : per) * blocks;
      quantize_rows_kernel<TYPE, VN><<<(unsigned)((total + 15) / 16), 256, 0, s>>>(x + r * n, n, blocks, total,
                                                                                 codes + r * n, scales + r * blocks);
      MOE_HIP(hipGetLastError());
    }
    return MOE_OK;
  }
  const int row_blocks = (rows + kBlock - 1) / kBlock;
  const long total = count * row_blocks * blocks;
  for (long b = 0; b < total; b += kMaxBlocks) {
    const long c = total - b < kMaxBlocks ? total - b : kMaxBlocks;
    quantize_blocks_kernel<TYPE, VN><<<(unsigned)c, 256, 0, s>>>(x, rows, n, row_blocks, blocks, b, codes, scales);
    MOE_HIP(hipGetLastError());
  }
  return MOE_OK;
}
template <int TYPE>
int quantize_typed(const void* x, long count, int rows, int n, int block_rows, uint8_t* codes, float* scales,
                   hipStream_t s) {
  return n % 8 == 0 && aligned(x, 16) && aligned(codes, 8)
             ? quantize<TYPE, 8>(x, count, rows, n, block_rows, codes, scales, s)
             : quantize<TYPE, 1>(x, count, rows, n, block_rows, codes, scales, s);
}

// ---------------------------------------------------------------- products
struct Fp8Args {
  const uint8_t* w;
  uint64_t w_stride;            // bytes from expert to expert
  const float* w_scales;
  uint64_t w_scales_stride;     // floats
  const uint8_t* x;
  const float* x_scales;
  int n_in, n_out, blocks;      // blocks of 128 inputs
  const int32_t* offsets;
  int E;
  long N;
  void* y;
  Grid grid;
};

// WQ x WP waves of TQ x TP tiles of 32 x 32, 128 inputs a step: a row's 128
// bytes lie in LDS as 64 elements of 16 bits do in tiles.h.
// Measured: 4096 rows, 4096 -> 16384 316 us (1740 TFLOP/s; 374 in the first
// launches on an idle card) with 256 x 256 a block: by the sums' 16 scaled
// additions a tile and step beside the products, and each step's barrier; 32768
// rows of 256 experts, 2048 -> 512 96 us with 128 x 128: by HBM (370 MB) and
// half-filled chunks.
template <int WQ_, int WP_, int TQ_, int TP_, int NS_> struct Fp8Shape {
  static constexpr int WQ = WQ_, WP = WP_, TQ = TQ_, TP = TP_, NS = NS_;
  // Scales are 2^-105 and larger, so that the product of two may leave fp32's range
  // while y does not (x and W of 2^-70), whereas a step's sum times one scale stays
  // above 2^-123 (nonzero products of codes are 2^-18 and larger).  With one tile a
  // wave each sum is scaled by the one and then by the other; with more, where 16
  // products a tile count, the scales are multiplied first and steps whose product
  // is no normal number come after the loop (us, one after the other and this: 300
  // x 4096 -> 4096, 64 x 64, 21.1 and 23.4; 500 x 4096 -> 16384, 128 x 128, 46.5 and
  // 43.0; 4096 x 4096 -> 16384, 256 x 256, 373 and 353, with the range left open 347;
  // where every step is such a one 2570, where sizes are filled up with zeros 360).
  static constexpr bool TWICE = TQ_ * TP_ == 1;
  static constexpr int NT = 64 * WQ * WP, BQ = 32 * WQ * TQ, BP = 32 * WP * TP;
  typedef Tile<true, BQ, 64, NT, false> QT;
  typedef Tile<true, BP, 64, NT, false> PT;
  static constexpr int kStage = QT::kBytes + PT::kBytes, kStages = NS * kStage;
};

template <class T> __device__ __forceinline__ i32x8_t fp8_frag(const uint8_t* t, int r0, int half, int lane) {
  const int row = r0 + (lane & 31), piece = 4 * half + 2 * (lane >> 5);
  const u32x4_t a = *reinterpret_cast<const u32x4_t*>(t + T::pos(row, piece));
  const u32x4_t b = *reinterpret_cast<const u32x4_t*>(t + T::pos(row, piece + 1));
  return (i32x8_t){(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// The K loop, for the first LIVE of the wave's tiles of x (a constant, as in
// tiles.h).  A row tile's fragments are read while the products of the one
// before run; each pair of products is folded into its sums meanwhile.
// Steps that are left out (S::TWICE) lie from `first` to `last`.
template <class S, int LIVE>
__device__ __forceinline__ void fp8_loop(const Operand& q, const Operand& p, uint8_t* lds, int blocks, const float* const (&sx)[S::TQ],
                                         const float* const (&sw)[S::TP], f32x16_t (&acc)[S::TQ][S::TP], int& first, int& last) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wq = wave / S::WP, wp = wave % S::WP;
  typename S::QT qt;
  typename S::PT pt;
  qt.plan(q);
  pt.plan(p);
  constexpr int kDma = S::QT::kPer + S::PT::kPer;
  const uint32_t base = lds_address(lds);
  const auto issue = [&](int s, uint32_t st) {
    const int k0 = s < blocks ? s * 64 : q.K;
    qt.dma(q, base + st, k0);
    pt.dma(p, base + st + S::QT::kBytes, k0);
  };
#pragma unroll
  for (int s = 0; s < S::NS - 1; ++s) issue(s, s * S::kStage);
  uint32_t now = 0, fill = (S::NS - 1) * S::kStage;             // stages, as bytes
  const auto after = [](uint32_t st) { return st == (S::NS - 1) * S::kStage ? 0 : st + S::kStage; };
  for (int s = 0; s < blocks; ++s) {
    bool all = true;
    float fx[LIVE + 1], fw[S::TP];
#pragma unroll
    for (int t = 0; t < LIVE; ++t) fx[t] = sx[t][s];
#pragma unroll
    for (int t = 0; t < S::TP; ++t) fw[t] = sw[t][s];
    stage_wait<(S::NS - 2) * kDma>();
    issue(s + S::NS - 1, fill);
    const uint8_t* st = lds + now;
    now = after(now);
    fill = after(fill);
    if constexpr (LIVE > 0) {
      i32x8_t pf[S::TP][2], qf[2][2];
      const auto read = [&](int u) {
#pragma unroll
        for (int h = 0; h < 2; ++h) qf[u & 1][h] = fp8_frag<typename S::QT>(st, 32 * (wq * S::TQ + u), h, lane);
      };
#pragma unroll
      for (int t = 0; t < S::TP; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) pf[t][h] = fp8_frag<typename S::PT>(st + S::QT::kBytes, 32 * (wp * S::TP + t), h, lane);
      read(0);
#pragma unroll
      for (int u = 0; u < LIVE; ++u) {
        if (u + 1 < LIVE) read(u + 1);
#pragma unroll
        for (int t = 0; t < S::TP; ++t) {
          f32x16_t part{};
          part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(pf[t][0], qf[u & 1][0], part, 0, 0, 0, 0, 0, 0);
          part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(pf[t][1], qf[u & 1][1], part, 0, 0, 0, 0, 0, 0);
          if constexpr (S::TWICE) {
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[u][t][i] = fmaf(fx[u] * part[i], fw[t], acc[u][t][i]);
            continue;
          }
          const float both = fx[u] * fw[t];
          const bool normal = __builtin_amdgcn_classf(both, kNormal);
          const float f = normal ? both : 0.f;
          all &= normal;
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[u][t][i] = fmaf(f, part[i], acc[u][t][i]);
        }
      }
    }
    if (!S::TWICE && __ballot(!all) != 0) {
      first = s < first ? s : first;
      last = s;
    }
  }
}

// Inputs k .. k + 31 of a row of n in memory, zeros past its end.
__device__ __forceinline__ i32x8_t fp8_inputs(const uint8_t* row, int k, int n) {
  i32x8_t v{};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (k + 16 * h < n) {
      const u32x4_t q = *reinterpret_cast<const u32x4_t*>(row + k + 16 * h);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] = (int)q[i];
    }
  return v;
}
// The steps that fp8_loop left out of 32 rows by 32 columns, from first to last:
// each sum is scaled by one scale and then by the other.  x, w: the lane's rows of
// the operands.  Straight from memory, and past steps where W is zeros: what is left
// out is mostly sizes filled up with zeros, whose scales are the smallest.
__device__ __forceinline__ void fp8_left_out(const uint8_t* x, const uint8_t* w, int n, int first, int last, const float* sx,
                                             const float* sw, f32x16_t& acc) {
  for (int s = first; s <= last; ++s) {
    const float fx = sx[s], fw = sw[s];
    const bool far = !__builtin_amdgcn_classf(fx * fw, kNormal);
    const int k = kBlock * s + 32 * ((threadIdx.x & 63) >> 5);
    const i32x8_t p0 = fp8_inputs(w, k, n), p1 = fp8_inputs(w, k + 64, n);
    int any = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= p0[i] | p1[i];
    if (__ballot(far) == 0 || __ballot((any & 0x7F7F7F7F) != 0 || !__builtin_isfinite(fw) || !__builtin_isfinite(fx)) == 0)
      continue;
    f32x16_t part{};
    part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(p0, fp8_inputs(x, k, n), part, 0, 0, 0, 0, 0, 0);
    part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(p1, fp8_inputs(x, k + 64, n), part, 0, 0, 0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = far ? fmaf(fx * part[i], fw, acc[i]) : acc[i];
  }
}

template <class S, int OUT>
__global__ __launch_bounds__(S::NT, 2) void linear_fp8_kernel(Fp8Args a) {
  extern __shared__ uint8_t tile_lds[];
  static_assert(S::NT / 64 * kTurn<OUT, S::TP> <= kBlockLds<S, OUT> && kBlockLds<S, OUT> <= kMaxLds, "turns in LDS");
  constexpr int kSize = El<OUT>::kN == 4 ? 4 : 2;
  int unit, tile;
  if (!grid_place(a.grid, &unit, &tile)) return;
  long start;
  int n, e = 0;
  if (a.offsets) {
    const RowChunk c = find_chunk(a.offsets, nullptr, a.E, a.N, unit, S::BQ);
    if (!c.any || c.n == 0) return;
    start = c.start;
    n = c.n;
    e = c.slot;
  } else {
    start = (long)unit * S::BQ;
    n = a.N - start < S::BQ ? (int)(a.N - start) : S::BQ;
  }
  const int p0 = tile * S::BP, cols = a.n_out - p0 < S::BP ? a.n_out - p0 : S::BP;
  Operand q{}, p{};
  q.base = a.x + start * a.n_in;
  p.base = a.w + (uint64_t)e * a.w_stride + (uint64_t)p0 * a.n_in;
  q.ld = p.ld = q.K = p.K = a.n_in / 2;
  q.n = n;
  p.n = cols;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wq = wave / S::WP, wp = wave % S::WP;
  const int left = n - 32 * wq * S::TQ;
  const int live = left <= 0 ? 0 : left >= 32 * S::TQ ? S::TQ : (left + 31) / 32;
  const float* sx[S::TQ];
  const float* sw[S::TP];
#pragma unroll
  for (int t = 0; t < S::TQ; ++t) {
    const int r = 32 * (wq * S::TQ + t) + (lane & 31);
    sx[t] = a.x_scales + (start + (r < n ? r : n - 1)) * a.blocks;
  }
#pragma unroll
  for (int t = 0; t < S::TP; ++t) {
    const int o = p0 + 32 * (wp * S::TP + t);
    sw[t] = a.w_scales + (uint64_t)e * a.w_scales_stride + (uint64_t)((o < a.n_out ? o : a.n_out - 1) / kBlock) * a.blocks;
  }
  f32x16_t acc[S::TQ][S::TP] = {};
  int first = a.blocks, last = -1;
  if (live == S::TQ) {
    fp8_loop<S, S::TQ>(q, p, tile_lds, a.blocks, sx, sw, acc, first, last);
  } else if (S::TQ == 4 && live == 3) {
    fp8_loop<S, (S::TQ == 4 ? 3 : 0)>(q, p, tile_lds, a.blocks, sx, sw, acc, first, last);
  } else if (S::TQ == 4 && live == 2) {
    fp8_loop<S, (S::TQ == 4 ? 2 : 0)>(q, p, tile_lds, a.blocks, sx, sw, acc, first, last);
  } else if (S::TQ > 1 && live == 1) {
    fp8_loop<S, (S::TQ > 1 ? 1 : 0)>(q, p, tile_lds, a.blocks, sx, sw, acc, first, last);
  } else {
    fp8_loop<S, 0>(q, p, tile_lds, a.blocks, sx, sw, acc, first, last);
  }
  stage_wait<0>();
  if (!S::TWICE && first <= last) {
#pragma unroll
    for (int t = 0; t < S::TQ; ++t)
#pragma unroll
      for (int u = 0; u < S::TP; ++u) {
        const int r = 32 * (wq * S::TQ + t) + (lane & 31), o = p0 + 32 * (wp * S::TP + u) + (lane & 31);
        fp8_left_out(a.x + (start + (r < n ? r : n - 1)) * a.n_in,
                     a.w + (uint64_t)e * a.w_stride + (uint64_t)(o < a.n_out ? o : a.n_out - 1) * a.n_in, a.n_in, first, last,
                     sx[t], sw[u], acc[t][u]);
      }
  }
  uint8_t* mine = tile_lds + wave * kTurn<OUT, S::TP>;
#pragma unroll
  for (int t = 0; t < S::TQ; ++t) {
    if (t >= live) continue;
    const long r0 = start + 32 * (wq * S::TQ + t);
    const int c0 = 32 * S::TP * wp;
    store_rows<OUT, S::TP, false>(mine, acc[t], static_cast<uint8_t*>(a.y) + kSize * (r0 * a.n_out + p0 + c0), a.n_out,
                                  left - 32 * t < 32 ? left - 32 * t : 32, cols - c0);
  }
}

// Few rows (stream.h): a block of 16 RT columns of W by 16 NT rows, its waves
// take the blocks of 128 inputs in turn, U of them in flight.  Lane (m = lane &
// 15, b = lane >> 4) holds inputs 32 b .. + 31 of column m and of row m.
template <int RT, int NT, int NW, int U, int OUT>
__global__ __launch_bounds__(64 * NW) void stream_fp8_kernel(Fp8Args a) {
  constexpr int kTiles = RT * NT;
  __shared__ float red[NW * kTiles * 256];
  int unit, tile;
  if (!grid_place(a.grid, &unit, &tile)) return;
  const Rows rows = chunk_rows(a.offsets, a.E, a.N, unit, 16 * NT);
  if (rows.n == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int m = lane & 15, b = lane >> 4;
  const int p0 = tile * 16 * RT;
  const uint8_t* wp[RT];
  const float* sw[RT];
  const uint8_t* xp[NT];
  const float* sx[NT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int c = p0 + 16 * r + m < a.n_out ? p0 + 16 * r + m : a.n_out - 1;
    const int o = p0 + 16 * r < a.n_out ? p0 + 16 * r : a.n_out - 1;          // 16 columns share their scales
    wp[r] = a.w + (uint64_t)rows.e * a.w_stride + (uint64_t)c * a.n_in + 32 * b;
    sw[r] = a.w_scales + (uint64_t)rows.e * a.w_scales_stride + (uint64_t)(o / kBlock) * a.blocks;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const long q = rows.start + (16 * t + m < rows.n ? 16 * t + m : rows.n - 1);
    xp[t] = a.x + q * a.n_in + 32 * b;
    sx[t] = a.x_scales + q * a.blocks;
  }
  f32x4_t acc[RT][NT] = {};
  u32x4_t wv[U][RT][2], xv[U][NT][2];
  float fw[U][RT], fx[U][NT];
  // pieces past n_in: zeros (the first of the row is loaded instead)
  const auto piece = [&](const uint8_t* p, int s, int h) {
    const int k = kBlock * s + 16 * h;
    const bool in = k + 32 * b < a.n_in;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(in ? p + k : p - 32 * b);
    return in ? v : (u32x4_t){0, 0, 0, 0};
  };
  const auto load = [&](int u, int s) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      wv[u][r][0] = piece(wp[r], s, 0);
      wv[u][r][1] = piece(wp[r], s, 1);
      fw[u][r] = sw[r][s];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      xv[u][t][0] = piece(xp[t], s, 0);
      xv[u][t][1] = piece(xp[t], s, 1);
      fx[u][t] = sx[t][s];
    }
  };
  const auto join = [](const u32x4_t (&v)[2]) {
    return (i32x8_t){(int)v[0][0], (int)v[0][1], (int)v[0][2], (int)v[0][3], (int)v[1][0], (int)v[1][1], (int)v[1][2], (int)v[1][3]};
  };
  const auto compute = [&](int u) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const f32x4_t part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(wv[u][r]), join(xv[u][t]), (f32x4_t){}, 0, 0, 0, 0, 0, 0);
        // (one scale after the other, as Fp8Shape says; here memory bounds)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][t][i] = fmaf(fx[u][t] * part[i], fw[u][r], acc[r][t][i]);
      }
  };
  const int count = wave < a.blocks ? (a.blocks - wave + NW - 1) / NW : 0;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < count) load(u, wave + u * NW);
  int i = 0;
  for (; i + U <= count; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      __builtin_amdgcn_sched_barrier(0);
      compute(u);
      __builtin_amdgcn_sched_barrier(0);
      if (i + U + u < count) load(u, wave + (i + U + u) * NW);
    }
  }
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (i + u < count) compute(u);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) share_put<kTiles>(red, wave, r * NT + t, acc[r][t]);
  __syncthreads();
  typedef typename El<OUT>::raw raw;
  raw* out = static_cast<raw*>(a.y);
  for (int v = threadIdx.x; v < 16 * RT * 16 * NT; v += 64 * NW) {
    const int c = v % (16 * RT), q = v / (16 * RT), t = q / 16;
    if (q < rows.n && p0 + c < a.n_out)
      out[(rows.start + q) * a.n_out + p0 + c] = El<OUT>::down(share_sum<kTiles, NW>(red, (c / 16) * NT + t, q & 15, c & 15));
  }
}

template <int RT, int NT, int NW, int U, int OUT> int stream(Fp8Args& a, hipStream_t s) {
  const long units = a.offsets ? max_chunks(a.N, a.E, 16 * NT) : (a.N + 16 * NT - 1) / (16 * NT);
  return grid_launch(units, (a.n_out + 16 * RT - 1) / (16 * RT), 1, [&](const Grid& g, unsigned blocks) {
    a.grid = g;
    stream_fp8_kernel<RT, NT, NW, U, OUT><<<blocks, 64 * NW, 0, s>>>(a);
    MOE_HIP(hipGetLastError());
    return (int)MOE_OK;
  });
}

template <class S, int OUT> int tiled(Fp8Args& a, hipStream_t s) {
  const long units = a.offsets ? max_chunks(a.N, a.E, S::BQ) : (a.N + S::BQ - 1) / S::BQ;
  return grid_launch(units, (a.n_out + S::BP - 1) / S::BP, 4, [&](const Grid& g, unsigned blocks) {
    a.grid = g;
    linear_fp8_kernel<S, OUT><<<blocks, S::NT, kBlockLds<S, OUT>, s>>>(a);
    MOE_HIP(hipGetLastError());
    return (int)MOE_OK;
  });
}

template <int OUT> int product(Fp8Args& a, hipStream_t s) {
  // experts: tiles sooner than in 16 bits (us, streamed and in tiles, 2048 -> 512:
  // 160 rows of 512 experts 42 and 46, 320 79 and 75, 640 109 and 78)
  const int form = a.offsets && (a.N < a.E ? a.N : a.E) * ((a.n_out + 127) / 128) > 1024 ? 0 : few_rows(a.offsets ? a.E : 0, a.N);
  // waves that share the inputs (us: 2048 x 512, 10 rows of 512 experts: 8 waves
  // 6.0, 4 6.1, 2 6.8; 512 x 2048: 7.9, 7.1, 5.6; 1 row of 2048 x 100003 37.9,
  // 36.5, 39.5; of 4096 x 4096 6.4, 6.8, 9.3)
  if (form == 1 && a.blocks < 8) return stream<2, 1, 2, 4, OUT>(a, s);
  if (form == 1) return a.n_out >= 16384 ? stream<1, 1, 4, 4, OUT>(a, s) : stream<1, 1, 8, 2, OUT>(a, s);
  // more columns a block where there are many, as in product.hip
  if (form == 2) return a.n_out <= 8192 ? stream<1, 2, 8, 4, OUT>(a, s) : stream<2, 2, 4, 4, OUT>(a, s);
  if (form == 4) return a.n_out <= 8192 ? stream<1, 4, 8, 1, OUT>(a, s) : stream<2, 4, 4, 2, OUT>(a, s);
  if (few_tiles(a.offsets ? a.E : 0, a.N, a.n_out)) return tiled<Fp8Shape<2, 2, 1, 1, 5>, OUT>(a, s);
  if (wide_rows(a.offsets ? a.E : 0, a.N, a.n_out)) return tiled<Fp8Shape<2, 4, 4, 2, 2>, OUT>(a, s);
  return tiled<Fp8Shape<2, 2, 2, 2, 2>, OUT>(a, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_quantize_fp8(const void* x, int32_t type, int32_t count, int32_t rows, int32_t n,
                                int32_t block_rows, void* codes, float* scales, hipStream_t s) {
  MOE_CHECK(type_size(type) != 0 && count >= 0 && rows >= 0 && n >= 1 && (block_rows == 1 || block_rows == kBlock));
  if (n > kMostSize || (long)count * rows > (1l << 30)) return MOE_ERR_UNSUPPORTED;
  if (count == 0 || rows == 0) return MOE_OK;
  MOE_CHECK(x && codes && scales && aligned(x, type_size(type)) && aligned(scales, 4));
  uint8_t* c = static_cast<uint8_t*>(codes);
  if (type == MOE_TYPE_F32) return quantize_typed<MOE_TYPE_F32>(x, count, rows, n, block_rows, c, scales, s);
  return type == MOE_TYPE_BF16 ? quantize_typed<MOE_TYPE_BF16>(x, count, rows, n, block_rows, c, scales, s)
                               : quantize_typed<MOE_TYPE_F16>(x, count, rows, n, block_rows, c, scales, s);
}

extern "C" int moe_linear_fp8(const void* w, size_t w_stride, const float* w_scales, size_t w_scales_stride, int32_t E,
                              const void* x, const float* x_scales, int32_t N, int32_t n_in, int32_t n_out,
                              const int32_t* offsets, void* y, int32_t y_type, hipStream_t s) {
  MOE_TRY(product_check(E, MOE_TYPE_BF16, N, n_in, n_out, offsets));
  const long blocks = (n_in + kBlock - 1) / kBlock;
  MOE_CHECK(type_size(y_type) != 0 && n_in % 16 == 0 && aligned(w, 16) && w_stride % 16 == 0 && aligned(w_scales, 4));
  MOE_CHECK(E == 1 || (w_stride >= (size_t)n_in * n_out &&
                       w_scales_stride >= (size_t)blocks * ((n_out + kBlock - 1) / kBlock)));
  if (N == 0) return MOE_OK;
  MOE_CHECK(w && w_scales && x && x_scales && y && aligned(x, 16) && aligned(x_scales, 4) &&
            aligned(y, type_size(y_type)));
  Fp8Args a{};
  a.w = static_cast<const uint8_t*>(w);
  a.w_stride = w_stride;
  a.w_scales = w_scales;
  a.w_scales_stride = w_scales_stride;
  a.x = static_cast<const uint8_t*>(x);
  a.x_scales = x_scales;
  a.n_in = n_in;
  a.n_out = n_out;
  a.blocks = (int)blocks;
  a.offsets = offsets;
  a.E = E;
  a.N = N;
  a.y = y;
  if (y_type == MOE_TYPE_F32) return product<MOE_TYPE_F32>(a, s);
  return y_type == MOE_TYPE_BF16 ? product<MOE_TYPE_BF16>(a, s) : product<MOE_TYPE_F16>(a, s);
}
