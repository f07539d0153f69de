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
#include "internal.h"
#include "chunks.h"
#include "device.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

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
};

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

// A block: 16 RT weight rows times 16 NT rows of x, the inputs dealt to its
// waves in steps of 64 (32 with groups of 32) and joined through LDS in wave
// order.  Lane (m = lane & 15, kb = lane >> 4) holds weight row m and token m
// of each tile; in a step of 64 its codes are words 2 (kb >> 1) + {0, 1} of the
// 16-byte piece kb & 1, its activations the 16 inputs those words cover.
template <int GROUP, int NT, int RT, bool EXP>
__global__ __launch_bounds__(512) void linear_int4_kernel(LinArgs a) {
  constexpr int kStep = GROUP == 32 ? 32 : 64;
  constexpr int kM = kStep / 32;                // matrix instructions a step
  constexpr int kU = NT == 1 ? 4 : 2;           // steps in flight a wave
  extern __shared__ float red[];                // [waves][RT][NT][4][64]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int waves = blockDim.x >> 6;
  const int m = lane & 15, kb = lane >> 4;
  const int tiles = (a.n_out + 16 * RT - 1) / (16 * RT);
  const int steps = a.n_in / kStep;
  uint32_t mask = 0x00780078u, base = 0x41804180u;
  asm("" : "+s"(mask));
  asm("" : "+v"(base));
  const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, (u32x4_t){0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
  for (long item = blockIdx.x; item < a.chunks * tiles; item += gridDim.x) {
    const long chunk = item / tiles;
    const int tile = (int)(item - chunk * tiles);
    long start;
    int n;
    const uint8_t* w = a.w;
    bool missing = false;
    if (EXP) {
      const RowChunk rc = find_chunk<false>(a.offsets, a.E, a.N, chunk, 16 * NT, nullptr);
      if (rc.e < 0) return;                     // chunks only grow with the item
      start = rc.start;
      n = rc.n;
      const int slot = a.slot_table ? a.slot_table[rc.e] : rc.e;
      missing = slot < 0 || slot >= a.n_slots;
      if (missing) {
        if (threadIdx.x == 0 && a.err && n > 0) atomicOr(a.err, 1);
      } else {
        w += (uint64_t)slot * a.w_stride;
      }
    } else {
      start = chunk * 16 * NT;
      n = a.N - start < 16 * NT ? (int)(a.N - start) : 16 * NT;
    }
    const uint32_t* sb = reinterpret_cast<const uint32_t*>(w + (uint64_t)(a.n_in / 32) * a.n_out * 16);
    int row[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      row[r] = (tile * RT + r) * 16 + m;
      if (row[r] >= a.n_out) row[r] = a.n_out - 1;
    }
    f32x4_t acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[r][t] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    const int end = missing ? 0 : steps;
    for (int s0 = wave; s0 < end; s0 += waves * kU) {
      uint32_t q[kU][RT][kM], sc[kU][RT];
      u32x4_t xv[kU][NT][kM];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int s = s0 + u * waves < end ? s0 + u * waves : s0;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if (kM == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(
                w + ((uint64_t)(2 * s + (kb & 1)) * a.n_out + row[r]) * 16 + (kb >> 1) * 8);
            q[u][r][0] = v.x;
            q[u][r][kM - 1] = v.y;
          } else {
            q[u][r][0] = *reinterpret_cast<const uint32_t*>(w + ((uint64_t)s * a.n_out + row[r]) * 16 + kb * 4);
          }
          sc[u][r] = sb[(uint64_t)(s * kStep / GROUP) * a.n_out + row[r]];
        }
        const int at = kM == 2 ? s * 64 + 32 * (kb & 1) + 16 * (kb >> 1) : s * 32 + 8 * kb;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bool live = 16 * t + m < n;
#pragma unroll
          for (int j = 0; j < kM; ++j)
            xv[u][t][j] = live ? *reinterpret_cast<const u32x4_t*>(a.x + (size_t)(start + 16 * t + m) * a.n_in + at + 8 * j)
                               : (u32x4_t){0u, 0u, 0u, 0u};
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (s0 + u * waves < end) {
          bf16x8_t xa[NT][kM];
          f32x4_t xs[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            xs[t] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < kM; ++j) {
              xa[t][j] = pair_x(xv[u][t][j]);
              xs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[t][j], ones, xs[t], 0, 0, 0);
            }
          }
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const float sv = f16_to_f32(sc[u][r]), bv = fmaf(-16.f, sv, f16_to_f32(sc[u][r] >> 16));
            bf16x8_t wb[kM];
#pragma unroll
            for (int j = 0; j < kM; ++j) wb[j] = codes_bf16(q[u][r][j], mask, base);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              f32x4_t p = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = 0; j < kM; ++j) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[t][j], wb[j], p, 0, 0, 0);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[r][t][i] += fmaf(sv, p[i], bv * xs[t][i]);
            }
          }
        }
      }
    }
    __syncthreads();                            // the item before has been read
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[((wave * RT + r) * NT + t) * 256 + i * 64 + lane] = acc[r][t][i];
    __syncthreads();
    for (int v = threadIdx.x; v < RT * NT * 256; v += blockDim.x) {
      float sum = red[v];
      for (int q = 1; q < waves; ++q) sum += red[q * RT * NT * 256 + v];
      const int l = v & 63, i = (v >> 6) & 3, t = (v >> 8) % NT, r = (v >> 8) / NT;
      const int o = (tile * RT + r) * 16 + (l & 15), tok = 16 * t + 4 * (l >> 4) + i;
      if (o < a.n_out && tok < n) a.y[(size_t)(start + tok) * a.n_out + o] = sum;
    }
  }
}

constexpr unsigned kMaxBlocks = 1u << 20;

template <int GROUP, int NT, int RT, bool EXP>
int launch(const LinArgs& a, hipStream_t s) {
  const int steps = a.n_in / (GROUP == 32 ? 32 : 64);
  const int waves = steps >= 16 ? 8 : steps >= 4 ? 4 : 1;
  const long tiles = (a.n_out + 16 * RT - 1) / (16 * RT);
  const long items = a.chunks * tiles;
  const unsigned grid = (unsigned)(items < (long)kMaxBlocks ? items : (long)kMaxBlocks);
  const size_t lds = (size_t)waves * RT * NT * 256 * sizeof(float);
  linear_int4_kernel<GROUP, NT, RT, EXP><<<grid, 64 * waves, lds, s>>>(a);
  MOE_HIP(hipGetLastError());
  return MOE_OK;
}

template <int GROUP, bool EXP>
int by_rows(LinArgs a, hipStream_t s) {
  // rows a chunk: all of them for one matrix, the expected rows of a bucket for experts
  const long rows = EXP ? (a.N + a.E - 1) / a.E : a.N;
  const int nt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  a.chunks = EXP ? max_chunks(a.N, a.E, 16 * nt, false) : (a.N + 16 * nt - 1) / (16 * nt);
  return nt == 1 ? launch<GROUP, 1, 1, EXP>(a, s) : nt == 2 ? launch<GROUP, 2, 1, EXP>(a, s)
                                                            : launch<GROUP, 4, 1, EXP>(a, s);
}

template <bool EXP> int linear_launch(const LinArgs& a, int group, hipStream_t s) {
  return group == 32 ? by_rows<32, EXP>(a, s) : group == 64 ? by_rows<64, EXP>(a, s) : by_rows<128, EXP>(a, s);
}

bool linear_ok(const moe_linear_shape* sh) {
  return sh && (sh->group == 32 || sh->group == 64 || sh->group == 128) && sh->n_in >= sh->group &&
         sh->n_in % sh->group == 0 && sh->n_in <= 65536 && sh->n_out >= 1 && sh->n_out <= (1 << 24);
}
size_t codes_bytes(const moe_linear_shape* sh) { return (size_t)sh->n_in / 2 * sh->n_out; }

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
  if (shape_bits(&fs) != 4) return MOE_ERR_UNSUPPORTED;
  const moe_linear_shape sh{matrix == 2 ? fs.I : fs.d, matrix == 2 ? fs.d : fs.I, 64};
  // a blob's matrix is its codes followed by its (scale, bias) words: the layout of one packed matrix
  return expert_linear(&sh, v.slab + blob_layout(fs.d, fs.I, 4).m[matrix].codes, v.stride,
                       moe_pool_num_slots(pool), v.slot_table, v.E, x_sorted, N, offsets, y_sorted, v.err, s);
}
