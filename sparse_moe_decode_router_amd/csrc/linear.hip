// Products of bf16 activations with 4-bit affine group-quantised matrices: one
// matrix (moe_linear_int4), or one per expert over rows in expert order
// (moe_expert_linear_int4, moe_pool_linear_int4).
//
// MLX affine int4 (relationship-to-TurboFieldfare section of the Swiftlet
// pages): W[o][j] = s q + b per group of inputs, so a group's share of y[o] is
//     s sum(q x) + b sum(x) = s sum((16+q) x) + (b - 16 s) sum(x).
// 16 + q is a bf16 with the code in the top four mantissa bits (0x4180 | q<<3),
// so four shifts and four v_and_or_b32 turn a word of eight codes into a matrix
// operand; both sums run on v_mfma_f32_16x16x32_bf16 (tokens by weight rows;
// the second against ones), every product exact, and each group is folded into
// the running fp32 sum with its own scale.  The offset 16 is the smallest that
// bf16 allows, which keeps the cancellation between the two terms small.
//
// One row is bound by HBM where the matrix is large (2048 x 100003: 24.7 us,
// 4.7 TB/s) and by the launch and two dependent loads where it is small (2048 x
// 2048: 4.1 us); tens of rows by latency, too few waves for it (48 rows of 4096
// x 4096: 10.2 us; 1.5 waves a SIMD, 44 % of their cycles waiting, and W read
// and decoded for every 16 rows; L2 gives 5 TB/s there, 20 elsewhere);
// thousands by one wave a SIMD with each step's loads directly before its sums,
// and the codes decoded by every wave (4096 rows of 2048 x 8192: 299 us, 460
// TFLOP/s).
#include "internal.h"
#include "device.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

struct LinArgs {
  const uint8_t* w;             // codes, then (scale, bias); expert slots w_stride apart
  uint64_t w_stride;
  const int32_t* slot_table;    // [E], or null: expert e in slot e
  int32_t n_slots, E;
  int32_t* err;                 // or null
  const int32_t* offsets;       // [E+1] (experts)
  const uint16_t* x;            // [N][n_in]
  float* y;                     // [N][n_out]
  int32_t n_in, n_out;
  long N;                       // rows of x
  long chunks;                  // upper bound of row chunks
  long chunk0;                  // this launch's first one
  // a block: wr row groups of 16 RT weight rows times wk shares of the inputs,
  // one wave each, over `turns` tiles of 16 RT wr rows (1 where wk > 1)
  int32_t wr, wk, turns;
  int32_t size;                 // rows a chunk, at most 16 NT
};

// Sorted rows are cut into chunks of `size` that do not cross an expert's
// border, numbered in expert order.
struct RowChunk {
  bool any;     // false past the last chunk
  int slot;     // of its expert
  int start;    // first row
  int n;        // rows (0..size)
};

// Chunk j.  Every wave finds its own: borders and slots of all experts in
// coalesced loads, all in flight at once (lane l holds experts l, l + 64, ..),
// chunks counted by wave scans of 64 experts.  Offsets that do not describe N
// rows give no row outside them.
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
      const int rows = 64 * u + 63 < E || lane < E - 64 * u ? next - off[u] : 0;
      const int c = rows > 0 ? (int)((unsigned)(rows + size - 1) / (unsigned)size) : 0;
      const int incl = wave_scan(c) + before;
      const uint64_t past = __ballot((long)incl > j);
      if (past != 0) {
        const int owner = __ffsll((unsigned long long)past) - 1;
        const int skip = ((int)j - __builtin_amdgcn_readlane(incl - c, owner)) * size;
        const int left = __builtin_amdgcn_readlane(rows, owner) - skip;
        r = RowChunk{true, __builtin_amdgcn_readlane(slots[u], owner), __builtin_amdgcn_readlane(off[u], owner) + skip,
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

// Eight codes of a word as bf16 16 + q, pairs (q[u], q[u+4]), u = 0..3.
__device__ __forceinline__ bf16x8_t codes_bf16(uint32_t w, uint32_t mask, uint32_t base) {
  u32x4_t r;
  r[0] = ((w << 3) & mask) | base;
  r[1] = ((w >> 1) & mask) | base;
  r[2] = ((w >> 5) & mask) | base;
  r[3] = ((w >> 9) & mask) | base;
  return __builtin_bit_cast(bf16x8_t, r);
}
// Eight activations in memory order as the pairs (x[u], x[u+4]).
__device__ __forceinline__ bf16x8_t pair_x(u32x4_t v) {
  u32x4_t r;
  r[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
  r[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
  r[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
  r[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
  return __builtin_bit_cast(bf16x8_t, r);
}

// A wave: 16 RT weight rows times 16 NT rows of x over the steps kq, kq + wk,
// ... of 64 inputs (32 with groups of 32), U steps of loads in flight.  Lane
// (m = lane & 15, kb = lane >> 4) holds weight row m and token m of each tile;
// in a step of 64 it loads words 2 (kb >> 1) + {0, 1} of the 16-byte piece kb & 1
// and swaps rows of lanes so that it holds word kb of both, whose inputs are the
// 16 bytes kb of either half of a 128-byte line of x.  The wk waves that
// share rows are joined through LDS in order.
template <int GROUP, int NT, int RT, int U, bool EXP, bool XL>
__global__ __launch_bounds__(512) void linear_int4_kernel(LinArgs a) {
  constexpr int kStep = GROUP == 32 ? 32 : 64;
  constexpr int kM = kStep / 32;                // matrix instructions a step
  static_assert(!XL || NT == 1, "x in LDS: one tile of tokens");
  extern __shared__ float red[];                // [waves][RT][NT][4][64] where wk > 1 | XL: x
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wr = wave / a.wk, kq = wave - wr * a.wk;
  const int m = lane & 15, kb = lane >> 4;
  const int rows = 16 * RT * a.wr;              // of a tile
  const int tiles = (a.n_out + rows - 1) / rows;
  const int tile_blocks = (tiles + a.turns - 1) / a.turns;
  const int steps = a.n_in / kStep;
  uint32_t mask = 0x00780078u, base = 0x41804180u;
  asm("" : "+s"(mask));
  asm("" : "+v"(base));
  const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, (u32x4_t){0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
  const long chunk = a.chunk0 + blockIdx.x / tile_blocks;
  const int tile0 = (int)(blockIdx.x % tile_blocks) * a.turns;
  long start;
  int n;
  const uint8_t* w = a.w;
  bool missing = false;
  if (EXP) {
    const RowChunk rc = find_chunk(a.offsets, a.slot_table, a.E, a.N, chunk, a.size);
    if (!rc.any) return;                        // past the last chunk
    if (rc.n == 0) return;                      // rows that x does not have
    start = rc.start;
    n = rc.n;
    const int slot = rc.slot;
    missing = slot < 0 || slot >= a.n_slots;
    if (missing) {
      if (threadIdx.x == 0 && a.err) atomicOr(a.err, 1);
    } else {
      w += (uint64_t)slot * a.w_stride;
    }
  } else {
    start = chunk * a.size;
    n = a.N - start < a.size ? (int)(a.N - start) : a.size;
  }
  const uint32_t sb0 = (uint32_t)(a.n_in / 32) * (uint32_t)a.n_out * 16u;
  const rsrc_t mr = make_rsrc(w, sb0 + (uint32_t)(a.n_in / GROUP) * (uint32_t)a.n_out * 4u);
  const int end = missing ? 0 : steps;
  // rows of x past the chunk read zeros from past the end of the buffer
  const rsrc_t xr = make_rsrc(a.x + (size_t)start * a.n_in, (uint32_t)(n * a.n_in) * 2u);
  const int x_lane = (m * a.n_in + 8 * kb) * 2;
  // XL: x in LDS as operands, rows 16 bytes more than n_in apart (16 rows on 16
  // banks of four), lanes past the chunk on its last row
  uint8_t* xl = reinterpret_cast<uint8_t*>(red + (a.wk > 1 ? a.wr * a.wk * RT * NT * 256 : 0));
  const uint32_t xl_lane = (uint32_t)((m < n ? m : n - 1) * (2 * a.n_in + 16) + 16 * kb);
  constexpr int kXP = 2;                        // pieces a thread loads before the weights
  const int x_pieces = n * (a.n_in / 8);
  u32x4_t xp[kXP];
  auto load_piece = [&](int p) {
    return __builtin_amdgcn_raw_buffer_load_b128(xr, p * 16, 0, 0);
  };
  auto store_piece = [&](int p, u32x4_t v) {
    const int t = p / (a.n_in / 8), c = p - t * (a.n_in / 8);
    *reinterpret_cast<bf16x8_t*>(xl + t * (2 * a.n_in + 16) + 16 * c) = pair_x(v);
  };
  if (XL) {
#pragma unroll
    for (int u = 0; u < kXP; ++u)
      if (threadIdx.x + u * blockDim.x < x_pieces) xp[u] = load_piece(threadIdx.x + u * blockDim.x);
  }
  for (int turn = 0; turn < a.turns && tile0 + turn < tiles; ++turn) {
    const int row0 = ((tile0 + turn) * a.wr + wr) * 16 * RT;
    uint32_t q_lane[RT], sb_lane[RT];         // byte offsets within a step's codes, a group's scales
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int row = row0 + 16 * r + m < a.n_out ? row0 + 16 * r + m : a.n_out - 1;
      q_lane[r] = kM == 2 ? (uint32_t)((kb & 1) * a.n_out + row) * 16u + (kb >> 1) * 8 : (uint32_t)row * 16u + kb * 4;
      sb_lane[r] = (uint32_t)row * 4u;
    }
    f32x4_t acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[r][t] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    uint32_t q[U][RT][kM], sc[U][RT];
    u32x4_t xv[XL ? 1 : U][NT][kM];
    auto load = [&](int u, int s) {
      const int qs = (int)((uint32_t)s * (uint32_t)(kStep / 2) * (uint32_t)a.n_out);
      const int ss = (int)(sb0 + (uint32_t)(s * kStep / GROUP) * (uint32_t)a.n_out * 4u);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if constexpr (kM == 2) {
          const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(mr, q_lane[r], qs, 0);
          q[u][r][0] = v[0];
          q[u][r][kM - 1] = v[1];
        } else {
          q[u][r][0] = __builtin_amdgcn_raw_buffer_load_b32(mr, q_lane[r], qs, 0);
        }
        sc[u][r] = __builtin_amdgcn_raw_buffer_load_b32(mr, sb_lane[r], ss, 0);
      }
      if constexpr (!XL) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < kM; ++j)
            xv[u][t][j] = __builtin_amdgcn_raw_buffer_load_b128(xr, x_lane + 16 * t * a.n_in * 2, s * kStep * 2 + 64 * j, 0);
      }
    };
    auto compute = [&](int u, int s) {
      bf16x8_t xa[NT][kM];
      f32x4_t xs[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        xs[t] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kM; ++j) {
          if constexpr (XL)
            xa[t][j] = *reinterpret_cast<const bf16x8_t*>(xl + xl_lane + s * kStep * 2 + 64 * j);
          else
            xa[t][j] = pair_x(xv[u][t][j]);
          xs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[t][j], ones, xs[t], 0, 0, 0);
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float sv = f16_to_f32(sc[u][r]), bv = fmaf(-16.f, sv, f16_to_f32(sc[u][r] >> 16));
        if constexpr (kM == 2) {                // word kb of piece 0, of piece 1
          const auto v = __builtin_amdgcn_permlane16_swap(q[u][r][0], q[u][r][1], false, false);
          q[u][r][0] = v[0];
          q[u][r][1] = v[1];
        }
        bf16x8_t wb[kM];
#pragma unroll
        for (int j = 0; j < kM; ++j) wb[j] = codes_bf16(q[u][r][j], mask, base);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          f32x4_t p = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < kM; ++j) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[t][j], wb[j], p, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][t][i] = fmaf(sv, p[i], fmaf(bv, xs[t][i], acc[r][t][i]));
        }
      }
    };
    const int count = kq < end ? (end - kq + a.wk - 1) / a.wk : 0;
    auto step = [&](int i) { return kq + i * a.wk; };
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < count) load(u, step(u));
    if (XL && turn == 0) {
#pragma unroll
      for (int u = 0; u < kXP; ++u)
        if (threadIdx.x + u * blockDim.x < x_pieces) store_piece(threadIdx.x + u * blockDim.x, xp[u]);
      for (int p = threadIdx.x + kXP * blockDim.x; p < x_pieces; p += blockDim.x) store_piece(p, load_piece(p));
      __syncthreads();
    }
    int i = 0;
    for (; i + U <= count; i += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // the compiler would otherwise gather the loads behind all the sums
        __builtin_amdgcn_sched_barrier(0);
        compute(u, step(i + u));
        __builtin_amdgcn_sched_barrier(0);
        if (i + U + u < count) load(u, step(i + U + u));
      }
    }
#pragma unroll
    for (int u = 0; u < U - 1; ++u)
      if (i + u < count) compute(u, step(i + u));
    if (a.wk == 1) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int o = row0 + 16 * r + m, tok = 16 * t + 4 * kb + i;
            if (o < a.n_out && tok < n) a.y[(size_t)(start + tok) * a.n_out + o] = acc[r][t][i];
          }
      continue;
    }
    __syncthreads();                          // the item before has been read
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[((wave * RT + r) * NT + t) * 256 + i * 64 + lane] = acc[r][t][i];
    __syncthreads();
    for (int v = threadIdx.x; v < a.wr * RT * NT * 256; v += blockDim.x) {
      const int g = v / (RT * NT * 256), z = v - g * (RT * NT * 256);
      const float* p = red + (size_t)g * a.wk * (RT * NT * 256) + z;
      float sum = p[0];
      for (int j = 1; j < a.wk; ++j) sum += p[j * (RT * NT * 256)];
      const int l = z & 63, i = (z >> 6) & 3, t = (z >> 8) % NT, r = (z >> 8) / NT;
      const int o = ((tile0 + turn) * a.wr + g) * 16 * RT + 16 * r + (l & 15), tok = 16 * t + 4 * (l >> 4) + i;
      if (o < a.n_out && tok < n) a.y[(size_t)(start + tok) * a.n_out + o] = sum;
    }
  }
}

inline size_t x_lds_bytes(int rows, int n_in) { return (size_t)rows * (2 * n_in + 16); }

constexpr long kMaxBlocks = 1l << 21;           // of a launch (its threads are counted in 32 bits)

template <int GROUP, int NT, int RT, int U, bool EXP, bool XL>
int launch(LinArgs a, int wk, long likely, hipStream_t s) {
  const int steps = a.n_in / (GROUP == 32 ? 32 : 64);
  a.wk = wk;
  while (a.wk > 1 && 4 * a.wk > steps) a.wk /= 2;       // a share of four steps at least
  a.wr = a.wk >= 4 ? 1 : XL && !EXP ? 8 / a.wk : 4 / a.wk;
  const long tiles = (a.n_out + 16 * RT * a.wr - 1) / (16 * RT * a.wr);
  a.turns = EXP && a.wk == 1 && tiles * likely >= 2048 ? 2 : 1;
  const long tile_blocks = (tiles + a.turns - 1) / a.turns;
  const size_t lds = (a.wk > 1 ? (size_t)a.wr * a.wk * RT * NT * 256 * sizeof(float) : 0) +
                     (XL ? x_lds_bytes(a.N < a.size ? (int)a.N : a.size, a.n_in) : 0);
  const long per = kMaxBlocks / tile_blocks > 0 ? kMaxBlocks / tile_blocks : 1;        // chunks a launch
  for (a.chunk0 = 0; a.chunk0 < a.chunks; a.chunk0 += per) {
    const long c = a.chunks - a.chunk0 < per ? a.chunks - a.chunk0 : per;
    linear_int4_kernel<GROUP, NT, RT, U, EXP, XL><<<(unsigned)(c * tile_blocks), 64 * a.wr * a.wk, lds, s>>>(a);
    MOE_HIP(hipGetLastError());
  }
  return MOE_OK;
}

// Tile shapes by the number of 16 x 16 output tiles, about a block for each of
// the 256 CUs first.  A block reads its rows of x and of W once, so beyond that
// wider tiles save reads: x is re-read for every row tile (from L2), W for
// every 16 rows.  Measured, us:
//   4096 x 4096   T = 1: RT 1 5.6, RT 2 6.8    T = 32: RT 1 13, RT 2 8.6, RT 4 11.2
//                 T = 64: RT 2 13.2, RT 4 11.5   T = 1024: RT 4 94, NT 4 RT 4 76
//   2048 x 8192   T = 1: RT 2 5.1, RT 1 5.3      T = 64: RT 4 11.5
//   4096 x 16384  T = 8: RT 2 10.6, RT 4 11.4    T = 16: RT 2 13.2, RT 4 11.9
//   2048 x 100003, T = 1: RT 2 28.1, with x in LDS 24.5 (4.7 TB/s)
//   256 experts of 512 x 2048, 512 rows: RT 4 35.6, RT 2 37.2, with x in LDS 33.4
// x in LDS (where a block's rows of it fit 32 KB) takes its loads, a fifth of
// a wave's, off the path of the weights.
// Inputs are split over the waves of a block (8 shares where blocks are few, 4
// or none where they are many), which keeps more loads in flight per CU than
// more steps per wave: 2048 x 2048, T = 1: 4.3 with four shares, 5.1 with two.
template <int GROUP, bool EXP>
int by_rows(LinArgs a, hipStream_t s) {
  const long rows = EXP ? (a.N + a.E - 1) / a.E : a.N;          // expected of a bucket, for experts
  const long t16 = (a.n_out + 15) / 16;
  const auto chunks = [&](int size, bool most) -> long {
    if (!EXP) return (a.N + size - 1) / size;
    return most ? max_chunks(a.N, a.E, size) : (a.N < a.E ? a.N : (rows + size - 1) / size * a.E);
  };
  const long wide = chunks(64, false);
  if (rows > 32 && t16 / 4 * wide >= 256) {
    a.size = 64;
    a.chunks = chunks(64, true);
    return launch<GROUP, 4, 4, 1, EXP, false>(a, t16 / 4 * wide >= 1024 ? 1 : 4, wide, s);
  }
  // rows a chunk: 16, or fewer for experts with few rows where x then fits LDS
  // and is held there; smaller chunks only read the matrix of a full bucket
  // more often (64 tokens, 8 of 256 experts, Zipf 1: 4096 x 2048 131 us with 16
  // rows, 164 with 4, 4096 x 512 28.5 against 44.6; even routing 249 and 247)
  constexpr size_t kXlMax = 32768;
  const auto fits = [&](int size) { return x_lds_bytes(a.N < size ? (int)a.N : size, a.n_in) <= kXlMax; };
  a.size = 16;
  if (EXP)
    while (a.size > 4 && a.size >= 4 * rows && x_lds_bytes(a.size, a.n_in) > kXlMax) a.size /= 2;
  // (a few blocks only wait longer for it: ten expert rows 7.1 against 7.6)
  const bool xl = t16 * chunks(a.size, false) > 512 && fits(a.size);
  if (!xl) a.size = 16;
  a.chunks = chunks(a.size, true);
  const long likely = chunks(a.size, false), units = t16 * likely;
  if (xl && rows <= 8 && units > 4096) return launch<GROUP, 1, 2, EXP ? 3 : 2, EXP, true>(a, 1, likely, s);
  if (EXP && units > 16384)
    return xl ? launch<GROUP, 1, 4, 2, EXP, true>(a, 1, likely, s) : launch<GROUP, 1, 4, 2, EXP, false>(a, 1, likely, s);
  if (units > 512 && rows > 8) {
    const int wk = units > 8192 ? 1 : units > 1024 ? 4 : 8;
    return xl ? launch<GROUP, 1, 4, 2, EXP, true>(a, wk, likely, s) : launch<GROUP, 1, 4, 2, EXP, false>(a, wk, likely, s);
  }
  if (units > 256) {
    const int wk = units > 16384 ? 1 : units > 1024 ? 4 : 8;
    return xl ? launch<GROUP, 1, 2, 2, EXP, true>(a, wk, likely, s) : launch<GROUP, 1, 2, 2, EXP, false>(a, wk, likely, s);
  }
  if (a.n_in >= 4096) return launch<GROUP, 1, 1, 4, EXP, false>(a, 8, likely, s);
  return launch<GROUP, 1, 1, 2, EXP, false>(a, 4, likely, s);
}

template <bool EXP> int linear_launch(const LinArgs& a, int group, hipStream_t s) {
  return group == 32 ? by_rows<32, EXP>(a, s) : group == 64 ? by_rows<64, EXP>(a, s) : by_rows<128, EXP>(a, s);
}

size_t codes_bytes(const moe_linear_shape* sh) { return (size_t)sh->n_in / 2 * sh->n_out; }
// A matrix is read through 32-bit buffer offsets: below 4 GiB.
bool linear_ok(const moe_linear_shape* sh) {
  return sh && (sh->group == 32 || sh->group == 64 || sh->group == 128) && sh->n_in >= sh->group &&
         sh->n_in % sh->group == 0 && sh->n_in <= 65536 && sh->n_out >= 1 && sh->n_out <= (1 << 24) &&
         codes_bytes(sh) + (size_t)(sh->n_in / sh->group) * sh->n_out * 4 < (1ull << 32);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_linear_bytes(const moe_linear_shape* sh) {
  return linear_ok(sh) ? codes_bytes(sh) + (size_t)(sh->n_in / sh->group) * sh->n_out * 4 : 0;
}

extern "C" int moe_pack_linear_int4(const moe_linear_shape* sh, const uint8_t* codes, const uint16_t* scales,
                                    const uint16_t* biases, void* out) {
  MOE_CHECK(linear_ok(sh) && codes && scales && biases && out);
  const size_t n_in = sh->n_in, n_out = sh->n_out, G = sh->n_in / sh->group;
  for (size_t i = 0; i < n_in * n_out; ++i) MOE_CHECK(codes[i] <= 15);
  uint8_t* c = static_cast<uint8_t*>(out);
  uint8_t* sb = c + codes_bytes(sh);
  for (size_t o = 0; o < n_out; ++o) {
    for (size_t j = 0; j < n_in; j += 2)
      c[((j / 32) * n_out + o) * 16 + (j % 32) / 2] = (uint8_t)(codes[o * n_in + j] | (codes[o * n_in + j + 1] << 4));
    for (size_t g = 0; g < G; ++g) {
      uint8_t* p = sb + (g * n_out + o) * 4;
      const uint16_t s = scales[o * G + g], b = biases[o * G + g];
      p[0] = (uint8_t)s;
      p[1] = (uint8_t)(s >> 8);
      p[2] = (uint8_t)b;
      p[3] = (uint8_t)(b >> 8);
    }
  }
  return MOE_OK;
}

extern "C" int moe_unpack_linear_int4(const moe_linear_shape* sh, const void* packed, uint8_t* codes, uint16_t* scales,
                                      uint16_t* biases) {
  MOE_CHECK(linear_ok(sh) && packed && codes && scales && biases);
  const size_t n_in = sh->n_in, n_out = sh->n_out, G = sh->n_in / sh->group;
  const uint8_t* c = static_cast<const uint8_t*>(packed);
  const uint8_t* sb = c + codes_bytes(sh);
  for (size_t o = 0; o < n_out; ++o) {
    for (size_t j = 0; j < n_in; ++j)
      codes[o * n_in + j] = (c[((j / 32) * n_out + o) * 16 + (j % 32) / 2] >> (4 * (j & 1))) & 15;
    for (size_t g = 0; g < G; ++g) {
      const uint8_t* p = sb + (g * n_out + o) * 4;
      scales[o * G + g] = (uint16_t)(p[0] | (p[1] << 8));
      biases[o * G + g] = (uint16_t)(p[2] | (p[3] << 8));
    }
  }
  return MOE_OK;
}

extern "C" int moe_linear_int4(const moe_linear_shape* sh, const void* w, const uint16_t* x, int32_t T, float* y,
                               hipStream_t s) {
  MOE_CHECK(linear_ok(sh) && T >= 0);
  if (T == 0) return MOE_OK;
  MOE_CHECK(w && x && y && aligned(w, 4) && aligned(x, 16) && aligned(y, 4));
  LinArgs a{};
  a.w = static_cast<const uint8_t*>(w);
  a.x = x;
  a.y = y;
  a.n_in = sh->n_in;
  a.n_out = sh->n_out;
  a.N = T;
  return linear_launch<false>(a, sh->group, s);
}

static int expert_linear(const moe_linear_shape* sh, const void* w, size_t w_stride, int32_t n_slots,
                         const int32_t* slot_table, int32_t E, const uint16_t* x, int32_t N, const int32_t* offsets,
                         float* y, int32_t* err, hipStream_t s) {
  MOE_CHECK(linear_ok(sh) && N >= 0 && E >= 1 && E <= 1024 && n_slots >= 1);
  MOE_CHECK(slot_table || n_slots >= E);
  MOE_CHECK(w_stride % 4 == 0 && w_stride >= moe_linear_bytes(sh));
  if (N == 0) return MOE_OK;
  if (N > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  MOE_CHECK(w && x && offsets && y && aligned(w, 4) && aligned(x, 16) && aligned(y, 4) && aligned(offsets, 4) &&
            aligned(slot_table, 4) && aligned(err, 4));
  LinArgs a{};
  a.w = static_cast<const uint8_t*>(w);
  a.w_stride = w_stride;
  a.slot_table = slot_table;
  a.n_slots = n_slots;
  a.E = E;
  a.err = err;
  a.offsets = offsets;
  a.x = x;
  a.y = y;
  a.n_in = sh->n_in;
  a.n_out = sh->n_out;
  a.N = N;
  return linear_launch<true>(a, sh->group, s);
}

extern "C" int moe_expert_linear_int4(const moe_linear_shape* sh, const void* w, size_t w_stride, int32_t n_slots,
                                      const int32_t* slot_table, int32_t E, const uint16_t* x_sorted, int32_t N,
                                      const int32_t* offsets, float* y_sorted, int32_t* error, hipStream_t s) {
  return expert_linear(sh, w, w_stride, n_slots, slot_table, E, x_sorted, N, offsets, y_sorted, error, s);
}

extern "C" int moe_pool_linear_int4(const moe_pool* pool, int32_t matrix, const uint16_t* x_sorted, int32_t N,
                                    const int32_t* offsets, float* y_sorted, hipStream_t s) {
  MOE_CHECK(pool && matrix >= 0 && matrix < 3);
  moe_ffn_shape fs;
  PoolView v;
  MOE_CHECK(pool_view(pool, &v) && pool_shape(pool, &fs));
  int dev = -1;
  MOE_HIP(hipGetDevice(&dev));
  MOE_CHECK(dev == v.device);                   // another device would read the pool's memory as its own
  if (shape_bits(&fs) != 4) return MOE_ERR_UNSUPPORTED;
  const moe_linear_shape sh{matrix == 2 ? fs.I : fs.d, matrix == 2 ? fs.d : fs.I, 64};
  // a blob's matrix is its codes followed by its (scale, bias) words: the layout of one packed matrix
  return expert_linear(&sh, v.slab + blob_layout(fs.d, fs.I, 4).m[matrix].codes, v.stride,
                       moe_pool_num_slots(pool), v.slot_table, v.E, x_sorted, N, offsets, y_sorted, v.err, s);
}
