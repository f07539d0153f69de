// Products of a few rows (16 NT of one expert, or of all) with 16-bit matrices:
// W goes from memory to the matrix cores' operands directly, each row of W read
// once by the one block that owns it, K shared by the waves of the block so
// that all of a block's loads are in flight together.  (rows_kernel's tiles
// would leave most CUs idle: 10 rows of 10 experts, 2048 -> 2 x 512, are 80
// tiles, 22.7 us; here 320 blocks, 12.1.)
//
// Bound by HBM where the matrices are many or large (64 tokens of 8 of 256
// experts, 2048 -> 2 x 512: 162 us, 5.8 TB/s; in e4m3 1 row, 2048 -> 100003:
// 34.3 us, 6.0 TB/s), by the launch and two dependent loads (borders, then rows
// and matrices) where they are few (10 rows of 10 experts, 512 -> 2048: 6.9 us
// for 21 MB).
#pragma once

#include <type_traits>

#include "tiles.h"

namespace moe {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
template <int TYPE> __device__ __forceinline__ f32x4_t mfma16(s16x8_t a, s16x8_t b, f32x4_t c) {
  if constexpr (TYPE == MOE_TYPE_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_v, a), __builtin_bit_cast(bf16x8_v, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_v, a), __builtin_bit_cast(f16x8_v, b), c, 0, 0, 0);
}

// The chunk of rows of a block.
struct Rows {
  long start;
  int n, e;                     // 0 rows: none
};
__device__ __forceinline__ Rows chunk_rows(const int32_t* offsets, int E, long N, int unit, int size) {
  Rows r{0, 0, 0};
  if (offsets) {
    const RowChunk c = find_chunk(offsets, nullptr, E, N, unit, size);
    if (c.any) r = Rows{c.start, c.n, c.slot};
  } else {
    r.start = (long)unit * size;
    r.n = N - r.start < size ? (int)(N - r.start) : size;
  }
  return r;
}

// The waves' partial sums of a block: [NW][tile of 16 x 16][i][lane], in LDS.
template <int TILES> __device__ __forceinline__ void share_put(float* red, int wave, int tile, f32x4_t v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) red[((wave * TILES + tile) * 4 + i) * 64 + (threadIdx.x & 63)] = v[i];
}
// Row q (of 16) and column p (of 16) of a tile, the shares added in order.
template <int TILES, int NW> __device__ __forceinline__ float share_sum(const float* red, int tile, int q, int p) {
  const float* at = red + (tile * 4 + (p & 3)) * 64 + (p >> 2) * 16 + q;
  float v = at[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) v += at[w * TILES * 256];
  return v;
}

// A block: 16 RT columns of W (GATED: 16 RT / 2 of each matrix, in turns of 16)
// by 16 NT rows; wave w takes steps w, w + NW, .. of 64 k, U of them in flight.
// Lane (m = lane & 15, b = lane >> 4) holds k 32 h + 8 b .. + 7 of column m and
// of row m.
template <int TYPE, bool GATED, int RT, int NT, int NW, int U, int OUT, bool AL>
__global__ __launch_bounds__(64 * NW) void stream_kernel(RowsArgs a) {
  constexpr int kTiles = RT * NT;
  typedef typename std::conditional<AL, u32x4_t, Piece16>::type Piece;
  __shared__ float red[NW * kTiles * 256];
  int unit, tile;
  if (!grid_place(a.grid, &unit, &tile)) return;
  const Rows rows = chunk_rows(a.offsets, a.E, a.N, unit, 16 * NT);
  if (rows.n == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int m = lane & 15, b = lane >> 4;
  constexpr int kCols = GATED ? 8 * RT : 16 * RT;
  const int p0 = tile * kCols;
  const uint8_t* w1 = a.p + (uint64_t)rows.e * a.p_stride;
  const uint8_t* w2 = GATED ? a.p2 + (uint64_t)rows.e * a.p2_stride : nullptr;
  // columns and rows that do not exist: the last one's, never stored
  const uint16_t* wp[RT];
  const uint16_t* xp[NT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int c = p0 + 16 * (GATED ? r / 2 : r) + m;
    wp[r] = reinterpret_cast<const uint16_t*>(GATED && (r & 1) ? w2 : w1) + (long)(c < a.P ? c : a.P - 1) * a.p_ld + 8 * b;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int q = 16 * t + m < rows.n ? 16 * t + m : rows.n - 1;
    xp[t] = reinterpret_cast<const uint16_t*>(a.q) + (rows.start + q) * a.q_ld + 8 * b;
  }
  f32x4_t acc[RT][NT] = {};
  const int steps = a.K / 64;
  u32x4_t wv[U][2][RT], xv[U][2][NT];
  const auto load = [&](int u, int s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int r = 0; r < RT; ++r) wv[u][h][r] = *reinterpret_cast<const Piece*>(wp[r] + 64l * s + 32 * h);
#pragma unroll
      for (int t = 0; t < NT; ++t) xv[u][h][t] = *reinterpret_cast<const Piece*>(xp[t] + 64l * s + 32 * h);
    }
  };
  const auto compute = [&](int u) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[r][t] = mfma16<TYPE>(__builtin_bit_cast(s16x8_t, wv[u][h][r]), __builtin_bit_cast(s16x8_t, xv[u][h][t]), acc[r][t]);
  };
  const int count = wave < steps ? (steps - wave + NW - 1) / NW : 0;
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
  // the k past whole steps
  if (64 * steps < a.K && wave == steps % NW) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 64 * steps + 32 * h;
#pragma unroll
      for (int r = 0; r < RT; ++r) wv[0][h][r] = load_piece(wp[r] - 8 * b, k + 8 * b, a.K);
#pragma unroll
      for (int t = 0; t < NT; ++t) xv[0][h][t] = load_piece(xp[t] - 8 * b, k + 8 * b, a.K);
    }
    compute(0);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) share_put<kTiles>(red, wave, r * NT + t, acc[r][t]);
  __syncthreads();
  typedef typename El<OUT>::raw raw;
  raw* out = static_cast<raw*>(a.out);
  for (int v = threadIdx.x; v < kCols * 16 * NT; v += 64 * NW) {
    const int c = v % kCols, q = v / kCols, t = q / 16;
    if (q >= rows.n || p0 + c >= a.P) continue;
    const long row = rows.start + q;
    if constexpr (GATED) {
      const float g = share_sum<kTiles, NW>(red, (2 * (c / 16)) * NT + t, q & 15, c & 15);
      const float u = share_sum<kTiles, NW>(red, (2 * (c / 16) + 1) * NT + t, q & 15, c & 15);
      out[row * a.P + p0 + c] = El<OUT>::down(act_value(a.act, g) * u);
      if (a.pre) {
        a.pre[2 * row * a.P + p0 + c] = g;
        a.pre[(2 * row + 1) * a.P + p0 + c] = u;
      }
    } else {
      out[row * a.P + p0 + c] = El<OUT>::down(share_sum<kTiles, NW>(red, (c / 16) * NT + t, q & 15, c & 15));
    }
  }
}

// Rows a chunk (the fewest, so that the matrices are read least often).
template <int TYPE, bool GATED, int RT, int NT, int NW, int U, int OUT, bool AL> int stream_launch(RowsArgs& a, hipStream_t s) {
  const long units = a.offsets ? max_chunks(a.N, a.E, 16 * NT) : (a.N + 16 * NT - 1) / (16 * NT);
  constexpr int kCols = GATED ? 8 * RT : 16 * RT;
  return grid_launch(units, (a.P + kCols - 1) / kCols, 1, [&](const Grid& g, unsigned blocks) {
    a.grid = g;
    stream_kernel<TYPE, GATED, RT, NT, NW, U, OUT, AL><<<blocks, 64 * NW, 0, s>>>(a);
    MOE_HIP(hipGetLastError());
    return (int)MOE_OK;
  });
}

}  // namespace moe
