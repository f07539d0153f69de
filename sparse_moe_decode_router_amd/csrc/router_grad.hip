// Gradient of the router (moe_router_topk): with the chosen experts e_r, their
// weights w (softmax over the chosen logits) and the shared gate s = sigmoid,
//     g[t,r] = w_r (dw_r - sum_j w_j dw_j),   g_s[t] = s (1 - s) ds
//     dx[t]  = sum_r g[t,r] W[e_r] + g_s[t] W[E]
//     dW[e]  = sum over the pairs of bucket e of g x[t],   dW[E] = sum_t g_s[t] x[t]
//     db[e]  = sum over the pairs of bucket e of g
// Only k + 1 of E + 1 logits of a token have a gradient, so both products are
// weighted sums of rows: dx gathers router rows per token, dW gathers token
// rows per bucket (the stable lists of moe_bucket_tokens), in chunks of kCP
// rows whose partial sums are joined in chunk order.  fp32 throughout, fixed
// order, no atomics.
#include "internal.h"
#include "chunks.h"
#include "device.h"

namespace moe {
namespace {

constexpr int kCols = 512;      // columns a block
constexpr int kCP = 64;         // rows a chunk
constexpr unsigned kMaxBlocks = 1u << 20;

inline unsigned capped(long n) { return (unsigned)(n < (long)kMaxBlocks ? n : (long)kMaxBlocks); }

// g [T][k+1] and dx; block = (token, kCols columns).
__global__ __launch_bounds__(128) void router_grad_x_kernel(
    const float* __restrict__ W, const int32_t* __restrict__ idx, const float* __restrict__ w,
    const float* __restrict__ sgate, const float* __restrict__ dw, const float* __restrict__ dsgate, int T, int d,
    int E, int k, float* __restrict__ g, float* __restrict__ dx) {
  extern __shared__ float lg[];                 // [k+1] g | [k+1] router row
  int* le = reinterpret_cast<int*>(lg + k + 1);
  const int tid = threadIdx.x, lane = tid & 63;
  const int slabs = dx ? (d + kCols - 1) / kCols : 1;
  for (long item = blockIdx.x; item < (long)T * slabs; item += gridDim.x) {
    const int t = (int)(item / slabs), slab = (int)(item % slabs);
    float z = 0.f;
    for (int r = lane; r < k; r += 64) z = fmaf(w[(size_t)t * k + r], dw[(size_t)t * k + r], z);
    z = wave_sum(z);
    __syncthreads();
    for (int r = tid; r <= k; r += 128) {
      float v = 0.f;
      int e = E;
      if (r < k) {
        const size_t i = (size_t)t * k + r;
        v = w[i] * (dw[i] - z);
        e = idx[i];
        if (e < 0 || e >= E) {                  // a pair without an expert
          v = 0.f;
          e = -1;
        }
      } else if (dsgate) {
        const float s = sgate[t];
        v = dsgate[t] * (s * (1.f - s));
      }
      lg[r] = v;
      le[r] = e;
      if (slab == 0) g[(size_t)t * (k + 1) + r] = v;
    }
    __syncthreads();
    const int c = slab * kCols + tid * 4;
    if (!dx || c >= d) continue;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kB = 8;
    for (int r0 = 0; r0 <= k; r0 += kB) {
      float4 v[kB];
      float gv[kB];
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        const int r = r0 + u <= k ? r0 + u : k;
        const int e = le[r];
        gv[u] = lg[r];
        v[u] = *reinterpret_cast<const float4*>(W + (size_t)(e < 0 ? 0 : e) * d + c);
      }
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        if (r0 + u <= k && le[r0 + u] >= 0) {
          acc.x = fmaf(gv[u], v[u].x, acc.x);
          acc.y = fmaf(gv[u], v[u].y, acc.y);
          acc.z = fmaf(gv[u], v[u].z, acc.z);
          acc.w = fmaf(gv[u], v[u].w, acc.w);
        }
      }
    }
    *reinterpret_cast<float4*>(dx + (size_t)t * d + c) = acc;
  }
}

// One chunk of a bucket (or of all tokens for row E), kCols columns: four
// waves take the chunk's rows in turn, joined in wave order.
__global__ __launch_bounds__(256) void router_grad_w_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ g, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ pair_ids, int T, int d, int E, int k, long chunks, float* __restrict__ dW,
    float* __restrict__ part, long part_rows) {
  __shared__ float red[4][8][64];
  __shared__ float lg[kCP];
  __shared__ int lt[kCP];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int slabs = (d + kCols - 1) / kCols;
  const long n = (long)T * k;
  for (long item = blockIdx.x; item < chunks * slabs; item += gridDim.x) {
    const long j = item / slabs;
    const int slab = (int)(item - j * slabs);
    ChunkTotals tot;
    RowChunk rc = find_chunk<true>(offsets, E, n, j, kCP, &tot);
    if (rc.e < 0) {                             // row E: the tokens themselves
      const long first = (j - tot.chunks) * kCP;
      if (first >= (T > 0 ? T : 1)) return;     // chunks only grow with the item
      rc.e = E;
      rc.start = (int)first;
      rc.n = T - first < kCP ? (int)(T - first) : kCP;
      rc.index = (int)(j - tot.chunks);
      rc.of = (T + kCP - 1) / kCP;              // no tokens: one chunk of none
      rc.multi = tot.multi;
    }
    __syncthreads();
    if (tid < kCP) {
      int t = 0;
      float v = 0.f;
      if (tid < rc.n) {
        if (rc.e == E) {
          t = rc.start + tid;
          v = g[(size_t)t * (k + 1) + k];
        } else {
          const int i = pair_ids[rc.start + tid];
          if (i >= 0 && i < n) {
            t = i / k;
            v = g[(size_t)i + t];
          }
        }
      }
      lt[tid] = t;
      lg[tid] = v;
    }
    __syncthreads();
    const int c = slab * kCols + lane * 8;
    const int cc = c < d ? c : d - 8;           // columns past the row: a piece that is not stored
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    constexpr int kB = 8;
    for (int q0 = wave; q0 < rc.n; q0 += 4 * kB) {
      uint4 v[kB];
      float gv[kB];
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        const int q = q0 + 4 * u < kCP ? q0 + 4 * u : kCP - 1;
        gv[u] = q0 + 4 * u < rc.n ? lg[q] : 0.f;
        v[u] = *reinterpret_cast<const uint4*>(x + (size_t)lt[q] * d + cc);
      }
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        if (q0 + 4 * u < rc.n) {
          const uint32_t p[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[2 * i] = fmaf(gv[u], bf16_lo(p[i]), acc[2 * i]);
            acc[2 * i + 1] = fmaf(gv[u], bf16_hi(p[i]), acc[2 * i + 1]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    if (rc.of > 1 && rc.multi + rc.index >= part_rows) continue;   // offsets that are not T k rows
    float* dst = rc.of > 1 ? part + (size_t)(rc.multi + rc.index) * d : dW + (size_t)rc.e * d;
    for (int o = tid; o < kCols; o += 256) {
      const int l = o >> 3, i = o & 7;
      const float v = ((red[0][i][l] + red[1][i][l]) + red[2][i][l]) + red[3][i][l];
      if (slab * kCols + o < d) dst[slab * kCols + o] = v;
    }
  }
}

// Chunk sums of the rows that have several, joined in order; db.  Block =
// (router row, kCols columns).
__global__ __launch_bounds__(128) void router_grad_join_kernel(
    const float* __restrict__ g, const int32_t* __restrict__ offsets, const int32_t* __restrict__ pair_ids, int T,
    int d, int E, int k, const float* __restrict__ part, long part_rows, float* __restrict__ dW, float* __restrict__ dbias) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int slabs = dW ? (d + kCols - 1) / kCols : 1;
  const long n = (long)T * k;
  for (int item = blockIdx.x; item < (E + 1) * slabs; item += gridDim.x) {
    const int e = item / slabs, slab = item % slabs;
    // chunks of multi-chunk experts before e, and of e itself
    int before = 0, mine = 0;
    for (int q = lane; q < E && q <= e; q += 64) {
      const int rows = offsets[q + 1] - offsets[q];
      const int c = rows > 0 ? (rows + kCP - 1) / kCP : 0;
      if (q < e) before += c > 1 ? c : 0;
    }
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) before += __shfl_xor(before, s, 64);
    if (e < E) {
      const int rows = offsets[e + 1] - offsets[e];
      mine = rows > 0 ? (rows + kCP - 1) / kCP : 0;
    } else {
      mine = (T + kCP - 1) / kCP;
    }
    const int c = slab * kCols + tid * 4;
    if (dW && mine > 1 && c < d && (long)before + mine <= part_rows) {
      const float* p = part + (size_t)before * d + c;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int kB = 8;
      for (int q0 = 0; q0 < mine; q0 += kB) {
        float4 v[kB];
#pragma unroll
        for (int u = 0; u < kB; ++u)
          v[u] = *reinterpret_cast<const float4*>(p + (size_t)(q0 + u < mine ? q0 + u : mine - 1) * d);
#pragma unroll
        for (int u = 0; u < kB; ++u) {
          if (q0 + u < mine) {
            acc.x += v[u].x; acc.y += v[u].y; acc.z += v[u].z; acc.w += v[u].w;
          }
        }
      }
      *reinterpret_cast<float4*>(dW + (size_t)e * d + c) = acc;
    }
    if (dbias && slab == 0 && e < E && tid < 64) {
      float v = 0.f;
      for (long q = (long)offsets[e] + lane; q < offsets[e + 1] && q >= 0 && q < n; q += 64) {
        const int i = pair_ids[q];
        if (i >= 0 && i < n) v += g[(size_t)i + i / k];
      }
      v = wave_sum(v);
      if (lane == 0) dbias[e] = v;
    }
  }
}

struct GradWs {
  float* g;
  float* part;
  long part_rows;
};
bool carve_grad(Carver& c, int T, int d, int E, int k, GradWs* w) {
  w->g = c.take<float>((size_t)T * (k + 1));
  // chunks of buckets that have more than one: rows <= T k make at most 2 T k / kCP of them
  w->part_rows = 2 * (long)T * k / kCP + (T + kCP - 1) / kCP + 1;
  w->part = c.take<float>((size_t)w->part_rows * d);
  return c.ok();
}
bool sizes_ok(int T, int d, int E, int k) {
  return T >= 0 && d >= 64 && d % 64 == 0 && d <= 8192 && E >= 1 && E <= 1024 && k >= 1 && k <= E &&
         (long)T * k <= (1L << 30);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_router_backward_workspace_bytes(int32_t T, int32_t d, int32_t E, int32_t k) {
  if (!sizes_ok(T, d, E, k)) return 0;
  Carver c(nullptr, (size_t)-1);
  GradWs w;
  carve_grad(c, T, d, E, k, &w);
  return c.off + 256;
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
  GradWs b{};
  if (T > 0) {
    Carver c(ws, ws_bytes);
    if (!carve_grad(c, T, d, E, k, &b)) return MOE_ERR_INVALID_ARG;
    const long slabs = dx ? (d + kCols - 1) / kCols : 1;
    router_grad_x_kernel<<<capped(T * slabs), 128, (size_t)(k + 1) * 8, s>>>(W, idx, w, sgate, dw, dsgate, T, d, E, k,
                                                                            b.g, dx);
    MOE_HIP(hipGetLastError());
  }
  if (dW) {
    const long slabs = (d + kCols - 1) / kCols;
    const long chunks = max_chunks((long)T * k, E, kCP, true) + (T > 0 ? (T + kCP - 1) / kCP : 1);
    router_grad_w_kernel<<<capped(chunks * slabs), 256, 0, s>>>(x, b.g, offsets, pair_ids, T, d, E, k, chunks, dW,
                                                               b.part, b.part_rows);
    MOE_HIP(hipGetLastError());
  }
  if (dW || dbias) {
    const long slabs = dW ? (d + kCols - 1) / kCols : 1;
    router_grad_join_kernel<<<capped((E + 1) * slabs), 128, 0, s>>>(b.g, offsets, pair_ids, T, d, E, k, b.part,
                                                                    b.part_rows, dW, dbias);
    MOE_HIP(hipGetLastError());
  }
  return MOE_OK;
}
