// Gradient of the router (moe_router_topk): with the chosen experts e_r, their
// weights w (softmax over the chosen logits) and the shared gate s = sigmoid,
//     g[t,r] = w_r (dw_r - sum_j w_j dw_j),   g_s[t] = s (1 - s) ds
//     dx[t]  = sum_r g[t,r] W[e_r] + g_s[t] W[E]
//     dW[e]  = sum over the pairs of bucket e of g x[t],   dW[E] = sum_t g_s[t] x[t]
//     db[e]  = sum over the pairs of bucket e of g
// A dropped pair (index outside [0, E)) is in no softmax: its w and dw, which
// may be anything, are in no sum (w is then the softmax over the others).
// Only k + 1 of E + 1 logits of a token have a gradient, so both products are
// weighted sums of rows: dx gathers router rows per token, dW gathers token
// rows per bucket (the stable lists of moe_bucket_tokens).  One launch, its
// blocks in three roles; fp32 throughout, fixed order, no atomics.  4096 tokens
// of 2048, 10 of 512 experts: 32 us with the pairs' launch, bound by the rows
// gathered through L2 (369 MB for dx, 184 MB for dW); three launches with
// partial sums joined in the last took 94.  64 tokens, 8 of 256: 5.0 us.
#include "internal.h"
#include "device.h"

namespace moe {
namespace {

// Threads a block: 512 keep fewer blocks of the expert rows on a CU (prompt of
// 4096 tokens 37.4 against 33.4 us, 64 tokens 8.7 against 5.5).
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kXCols = 256;     // columns a wave of the dx role
// Columns a block of the expert rows: 256 keep x's columns of an XCD in its L2
// for prompts (33.4 against 31.7 us), 512 make fewer blocks of few rows (5.3
// against 8.6).
constexpr int w_cols(bool prompt) { return prompt ? 256 : 512; }
constexpr int kECols = 64;      // columns a block of row E
// Up to this many pairs each role forms their g itself; more take a launch of
// their own first (4.6 us), which saves every column slab the k products of
// each pair (4096 tokens of 10: dW alone 29 against 36 us).
constexpr long kPairsMax = 4096;
// Blocks of the dx role in a launch (its threads are counted in 32 bits; 2^26
// tokens of 64 columns are 2^24 blocks).  A loop in the kernel instead cost a
// prompt 0.8 us.
constexpr unsigned kMaxXBlocks = 1u << 22;

struct GradArgs {
  const uint16_t* x;
  const float* W;
  const int32_t* idx;
  const float* w;
  const float* sgate;
  const float* dw;
  const float* dsgate;          // or null
  const int32_t* offsets;
  const int32_t* pair_ids;
  const float* g;               // [T][k+1], or null: formed where it is used
  float* dx;
  float* dW;
  float* dbias;
  int T, d, E, k;
  unsigned blocks_e, blocks_w;  // blocks of row E, of the expert rows; the rest: dx
  unsigned block0_x;            // this launch's first one of dx
};

__device__ __forceinline__ float gate_grad(const GradArgs& a, int t) {
  if (!a.dsgate) return 0.f;                    // its row of W is then not read either
  const float s = a.sgate[t];
  return a.dsgate[t] * (s * (1.f - s));
}

__device__ __forceinline__ bool has_logit(const GradArgs& a, int e) { return (unsigned)e < (unsigned)a.E; }
// v, or 0 whatever v holds (bits, so that no load of v waits behind the test).
__device__ __forceinline__ float keep_if(bool ok, float v) {
  return __uint_as_float(__float_as_uint(v) & (ok ? ~0u : 0u));
}

// g of pair i, which has a logit, of token t (one thread).
__device__ __forceinline__ float pair_grad(const GradArgs& a, long i, int t) {
  const float* w = a.w + (size_t)t * a.k;
  const float* dw = a.dw + (size_t)t * a.k;
  const int32_t* idx = a.idx + (size_t)t * a.k;
  constexpr int kB = 10;                        // loads in flight
  const float wi = a.w[i], di = a.dw[i];
  float z = 0.f;
  for (int r0 = 0; r0 < a.k; r0 += kB) {
    float u[kB], v[kB];
    int e[kB];
#pragma unroll
    for (int q = 0; q < kB; ++q) {
      const int r = r0 + q < a.k ? r0 + q : a.k - 1;
      u[q] = w[r];
      v[q] = dw[r];
      e[q] = idx[r];
    }
#pragma unroll
    for (int q = 0; q < kB; ++q) {
      const bool ok = r0 + q < a.k && has_logit(a, e[q]);
      z = fmaf(keep_if(ok, u[q]), keep_if(ok, v[q]), z);
    }
  }
  return wi * (di - z);
}

__global__ __launch_bounds__(256) void router_grad_pairs_kernel(GradArgs a, float* __restrict__ g) {
  const unsigned n = (unsigned)a.T * (unsigned)(a.k + 1);        // at most 2^29
  for (unsigned j = blockIdx.x * 256 + threadIdx.x; j < n; j += gridDim.x * 256) {
    const int t = (int)(j / (unsigned)(a.k + 1)), r = (int)(j % (unsigned)(a.k + 1));
    g[j] = r < a.k ? pair_grad(a, (long)t * a.k + r, t) : gate_grad(a, t);
  }
}

// acc[8] += gv * 8 bf16 of v
__device__ __forceinline__ void fma8(float (&acc)[8], float gv, uint4 v) {
  const uint32_t p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(gv, bf16_lo(p[i]), acc[2 * i]);
    acc[2 * i + 1] = fmaf(gv, bf16_hi(p[i]), acc[2 * i + 1]);
  }
}

// dW[E], kECols columns: groups of 8 lanes take the tokens in turn.
template <bool G>
__device__ void row_e(const GradArgs& a, int slab, float* red, float* lg) {
  constexpr int kB = 8, kG = kThreads / 8;
  const int tid = threadIdx.x, grp = tid >> 3;
  if (!a.dsgate) {                              // no gradient: zeros, whatever x and the gate hold
    if (tid < kECols) a.dW[(size_t)a.E * a.d + slab * kECols + tid] = 0.f;
    return;
  }
  const uint16_t* x = a.x + slab * kECols + (tid & 7) * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int t0 = 0; t0 < a.T; t0 += kG * kB) {
    uint4 v[kB];
#pragma unroll
    for (int u = 0; u < kB; ++u) {
      const int t = t0 + u * kG + grp;
      v[u] = *reinterpret_cast<const uint4*>(x + (size_t)(t < a.T ? t : a.T - 1) * a.d);
    }
    __syncthreads();
    if (t0 + tid < a.T) lg[tid] = G ? a.g[(size_t)(t0 + tid) * (a.k + 1) + a.k] : gate_grad(a, t0 + tid);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kB; ++u)
      if (t0 + u * kG + grp < a.T) fma8(acc, lg[u * kG + grp], v[u]);
  }
  static_assert(kG * kB == kThreads, "one weight a thread");
#pragma unroll
  for (int i = 0; i < 8; ++i) red[grp * 65 + (tid & 7) * 8 + i] = acc[i];
  __syncthreads();
  if (tid < kECols) {
    float v = 0.f;
    for (int q = 0; q < kG; ++q) v += red[q * 65 + tid];
    a.dW[(size_t)a.E * a.d + slab * kECols + tid] = v;
  }
}

// dW[e], kWCols columns (and db[e]): the waves take the bucket's pairs in turn.
template <bool G>
__device__ void row_expert(const GradArgs& a, int e, int slab, float* red, float* lg, int* lt) {
  constexpr int kB = 8, kTile = kThreads;       // pairs of a bucket at a time
  constexpr int kWCols = w_cols(G);
  constexpr int kL = kWCols / 8, kG = kThreads / kL;    // lanes a row, rows at once
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int grp = kL == 64 ? __builtin_amdgcn_readfirstlane(wave) : tid / kL;
  const long n = (long)a.T * a.k;
  long lo = a.offsets[e], hi = a.offsets[e + 1];
  lo = lo < 0 ? 0 : lo;                         // offsets of other pairs reach no memory past these
  hi = hi > n ? n : hi;
  const int c = slab * kWCols + tid % kL * 8;
  const uint16_t* x = a.x + (c < a.d ? c : a.d - 8);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float bias = 0.f;
  for (long p0 = lo; p0 < hi; p0 += kTile) {
    const int m = hi - p0 < kTile ? (int)(hi - p0) : kTile;
    __syncthreads();
    if (tid < m) {
      const int i = a.pair_ids[p0 + tid];
      const bool ok = i >= 0 && i < n;
      const int t = ok ? i / a.k : 0;
      const float g = !ok ? 0.f : G ? a.g[(size_t)i + t] : pair_grad(a, i, t);
      lt[tid] = t;
      lg[tid] = g;
      bias += g;
    }
    __syncthreads();
    if (a.dW) {
      for (int q0 = grp; q0 < m; q0 += kG * kB) {
        uint4 v[kB];
#pragma unroll
        for (int u = 0; u < kB; ++u)
          if (q0 + u * kG < m) {
            const int t = kL == 64 ? __builtin_amdgcn_readfirstlane(lt[q0 + u * kG]) : lt[q0 + u * kG];
            v[u] = *reinterpret_cast<const uint4*>(x + (size_t)t * a.d);
          }
#pragma unroll
        for (int u = 0; u < kB; ++u)
          if (q0 + u * kG < m) fma8(acc, lg[q0 + u * kG], v[u]);
      }
    }
  }
  if (a.dW) {
#pragma unroll
    for (int i = 0; i < 8; ++i) red[grp * kWCols + i * kL + tid % kL] = acc[i];
    __syncthreads();
    for (int o = tid; o < kWCols; o += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kG; ++q) v += red[q * kWCols + (o & 7) * kL + (o >> 3)];
      if (slab * kWCols + o < a.d) a.dW[(size_t)e * a.d + slab * kWCols + o] = v;
    }
  }
  if (a.dbias && slab == 0) {
    bias = wave_sum(bias);
    __syncthreads();
    if (lane == 0) lg[wave] = bias;
    __syncthreads();
    if (tid == 0) {
      float v = 0.f;
      for (int q = 0; q < kWaves; ++q) v += lg[q];
      a.dbias[e] = v;
    }
  }
}

// dx of one token, kXCols columns: one wave.
template <bool G>
__device__ void token_x(const GradArgs& a, int t, int slab) {
  constexpr int kB = 11;
  const int lane = threadIdx.x & 63;
  const int c = slab * kXCols + lane * 4;
  const float* W = a.W + (c < a.d ? c : a.d - 4);
  float z = 0.f;
  if (!G) {
    for (int r = lane; r < a.k; r += 64) {
      const size_t i = (size_t)t * a.k + r;
      const bool ok = has_logit(a, a.idx[i]);
      z = fmaf(keep_if(ok, a.w[i]), keep_if(ok, a.dw[i]), z);
    }
    z = wave_sum(z);
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r0 = 0; r0 <= a.k; r0 += 64) {       // 64 router rows' weights in the lanes
    const int r = r0 + lane;
    float gl = 0.f;
    int el = -1;
    if (r < a.k) {
      const size_t i = (size_t)t * a.k + r;
      el = has_logit(a, a.idx[i]) ? a.idx[i] : -1;
      gl = G ? a.g[i + t] : a.w[i] * (a.dw[i] - z);
    } else if (r == a.k) {
      el = a.dsgate ? a.E : -1;
      gl = G ? a.g[(size_t)t * (a.k + 1) + a.k] : gate_grad(a, t);
    }
    const int m = a.k + 1 - r0 < 64 ? a.k + 1 - r0 : 64;
    for (int q0 = 0; q0 < m; q0 += kB) {
      float4 v[kB];
      float gv[kB];
      int e[kB];
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        const int q = q0 + u < m ? q0 + u : m - 1;
        e[u] = q0 + u < m ? __builtin_amdgcn_readlane(el, q) : -1;
        gv[u] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gl), q));
        if (e[u] >= 0) v[u] = *reinterpret_cast<const float4*>(W + (size_t)e[u] * a.d);
      }
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        if (e[u] >= 0) {
          acc.x = fmaf(gv[u], v[u].x, acc.x);
          acc.y = fmaf(gv[u], v[u].y, acc.y);
          acc.z = fmaf(gv[u], v[u].z, acc.z);
          acc.w = fmaf(gv[u], v[u].w, acc.w);
        }
      }
    }
  }
  if (c < a.d) *reinterpret_cast<float4*>(a.dx + (size_t)t * a.d + c) = acc;
}

// Blocks of row E first (they take longest), then the expert rows, then dx.
// Blocks go to the 8 XCDs in turn, so numbering the column slabs fastest keeps
// one XCD's L2 on the same columns of x and W where their number divides 8.
// G: the pairs' g are in a.g.  Without, five waves a SIMD (90 registers; left
// alone the compiler takes 116, and the 1184 blocks of 64 tokens of 8 of 256,
// d = 2048, need a second round: 6.4 against 5.0 us).
template <bool G>
__global__ __launch_bounds__(kThreads, G ? 8 : 5) void router_grad_kernel(GradArgs a) {
  __shared__ float red[kThreads / 8 * 65];
  static_assert(kThreads / 8 * 65 >= kThreads * 8, "eight columns a thread");
  __shared__ float lg[kThreads];
  __shared__ int lt[kThreads];
  unsigned b = blockIdx.x;
  if (b < a.blocks_e) {
    row_e<G>(a, (int)b, red, lg);
    return;
  }
  b -= a.blocks_e;
  if (b < a.blocks_w) {
    const int slabs = a.dW ? (a.d + w_cols(G) - 1) / w_cols(G) : 1;
    row_expert<G>(a, (int)(b / slabs), (int)(b % slabs), red, lg, lt);
    return;
  }
  b -= a.blocks_w;
  b += a.block0_x;
  const int slabs = (a.d + kXCols - 1) / kXCols;
  const int t = (int)(b / slabs) * kWaves + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if (t < a.T) token_x<G>(a, t, (int)(b % slabs));
}

bool sizes_ok(int T, int d, int E, int k) {
  return T >= 0 && d >= 64 && d % 64 == 0 && d <= 8192 && E >= 1 && E <= 1024 && k >= 1 && k <= E &&
         (long)T * k <= (1L << 28) && (long)T * d <= (1L << 33);
}
size_t pairs_bytes(int T, int k) { return (size_t)T * (k + 1) * sizeof(float); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_router_backward_workspace_bytes(int32_t T, int32_t d, int32_t E, int32_t k) {
  if (!sizes_ok(T, d, E, k)) return 0;
  return pairs_bytes(T, k) + 256;
}

extern "C" int moe_router_topk_backward(const uint16_t* x, int32_t T, int32_t d, const float* W, int32_t E, int32_t k,
                                        const int32_t* idx, const float* w, const float* sgate, const float* dw,
                                        const float* dsgate, const int32_t* offsets, const int32_t* pair_ids,
                                        float* dx, float* dW, float* dbias, void* ws, size_t ws_bytes, hipStream_t s) {
  MOE_CHECK(sizes_ok(T, d, E, k));
  MOE_CHECK(dx || dW || dbias);
  MOE_CHECK((dW == nullptr && dbias == nullptr) || offsets);
  if (T > 0) {
    MOE_CHECK(x && W && idx && w && dw && ws && (dsgate == nullptr || sgate));
    MOE_CHECK((dW == nullptr && dbias == nullptr) || pair_ids);
  }
  MOE_CHECK(aligned(x, 16) && aligned(W, 16) && aligned(dx, 16) && aligned(dW, 16) && aligned(ws, 256));
  MOE_CHECK(T == 0 || ws_bytes >= pairs_bytes(T, k));
  GradArgs a{x, W, idx, w, sgate, dw, dsgate, offsets, pair_ids, nullptr, dx, dW, dbias, T, d, E, k, 0, 0, 0};
  if ((long)T * k > kPairsMax) {
    float* g = static_cast<float*>(ws);
    const long blocks = ((long)T * (k + 1) + 255) / 256;
    router_grad_pairs_kernel<<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, s>>>(a, g);
    MOE_HIP(hipGetLastError());
    a.g = g;
  }
  a.blocks_e = dW ? (unsigned)(d / kECols) : 0;
  const int cols = w_cols(a.g != nullptr);
  a.blocks_w = dW ? (unsigned)(E * ((d + cols - 1) / cols)) : dbias ? (unsigned)E : 0;
  const unsigned blocks_x = dx ? (unsigned)((T + kWaves - 1) / kWaves) * (unsigned)((d + kXCols - 1) / kXCols) : 0;
  do {
    const unsigned n = blocks_x - a.block0_x < kMaxXBlocks ? blocks_x - a.block0_x : kMaxXBlocks;
    const unsigned blocks = a.blocks_e + a.blocks_w + n;
    if (blocks == 0) return MOE_OK;             // dx of no tokens
    if (a.g)
      router_grad_kernel<true><<<blocks, kThreads, 0, s>>>(a);
    else
      router_grad_kernel<false><<<blocks, kThreads, 0, s>>>(a);
    MOE_HIP(hipGetLastError());
    a.blocks_e = a.blocks_w = 0;
    a.block0_x += n;
  } while (a.block0_x < blocks_x);
  return MOE_OK;
}
