// Token rows in expert order and back, with the gradients of both.
//
//   sort      X[row(i)] = x[t], i = t*k + r, row(i) = the pair's place in the
//             stable counting sort by expert (bucket.hip), -1 without one
//     grad    dx[t] = sum_r dX[row(t,r)]
//   unsort    y[t] = sum_r w[t,r] Y[row(t,r)] + s_t o[t]
//     grad    dY[row(t,r)] = w[t,r] dy[t],  dw[t,r] = <dy[t], Y[row(t,r)]>,
//             do[t] = s_t dy[t],  ds_t = <dy[t], o[t]>
//
// The batched and prefill passes of the Swiftlet layer ("How it works": k of E
// experts a token) group tokens by expert inside the library; these entry
// points give the rows themselves, for expert products of the caller's own.
// All sums run in fp32 in rank order (or a fixed tree over the columns), with
// no atomics, so results are bit-reproducible; each output is rounded once.
#include "internal.h"
#include "device.h"
#include "elem.h"

namespace moe {
namespace {

// Rows are cut into pieces of VN elements, one lane each.  The last piece of
// a row that VN does not divide starts VN before the row's end and repeats
// the elements it shares with the one before it (same values, same place).
template <int VN> __device__ __forceinline__ int piece_start(int c, int d) {
  const int e = c * VN;
  return e + VN <= d ? e : d - VN;
}

constexpr int kWaves = 4;                       // waves a block
constexpr unsigned kMaxBlocks = 1u << 22;       // blocks go round past this
constexpr long kMaxItems = (1l << 31) - 1;      // waves' work items, counted in 32 bits

inline unsigned wave_grid(long waves) {
  const long b = (waves + kWaves - 1) / kWaves;
  return (unsigned)(b < (long)kMaxBlocks ? b : (long)kMaxBlocks);
}

__device__ __forceinline__ long wave_id() {
  return (long)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}
__device__ __forceinline__ long wave_count() { return (long)gridDim.x * kWaves; }

// One wave per sorted row p: copy the token's row there and note the row at
// its pair; the wave also marks pair p if that pair has no expert.
template <int TYPE, int VN>
__global__ __launch_bounds__(64 * kWaves) void gather_rows_kernel(
    const typename El<TYPE>::raw* __restrict__ x, const int32_t* __restrict__ idx, long n, int k, int d, int E,
    const int32_t* __restrict__ offsets, const int32_t* __restrict__ pair_ids, int32_t* __restrict__ row_of,
    typename El<TYPE>::raw* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int pieces = (d + VN - 1) / VN;
  const int live = offsets[E];
  for (long p = wave_id(); p < n; p += wave_count()) {
    const int key = idx[p];
    if ((key < 0 || key >= E) && lane == 0) row_of[p] = -1;
    if (p >= live) continue;
    const int i = pair_ids[p];
    if (lane == 0) row_of[i] = (int32_t)p;
    const typename El<TYPE>::raw* src = x + (size_t)(i / k) * d;
    typename El<TYPE>::raw* dst = out + (size_t)p * d;
    for (int c = lane; c < pieces; c += 64) {
      const int e = piece_start<VN>(c, d);
      vec_store<TYPE, VN>(dst + e, vec_load<TYPE, VN>(src + e));
    }
  }
}

// The sort of a few decoded tokens (up to kFewMax pairs): a wave a pair, its
// place counted by ballots over all the keys, which the wave's lanes hold; no
// barrier.  offsets[e] counts the keys below e, a thread an entry.  One token
// of ten pairs: 2.7 us, 4.3 in sort_one_kernel.
constexpr int kFewMax = 256;
template <int TYPE, int VN>
__global__ __launch_bounds__(64 * kWaves) void sort_few_kernel(
    const typename El<TYPE>::raw* __restrict__ x, const int32_t* __restrict__ idx, int n, int k, int d, int E,
    int32_t* __restrict__ offsets, int32_t* __restrict__ pair_ids, int32_t* __restrict__ row_of,
    typename El<TYPE>::raw* __restrict__ out) {
  constexpr int kK = kFewMax / 64, kA = 4;
  const int tid = threadIdx.x, lane = tid & 63;
  const int i = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pieces = (d + VN - 1) / VN;
  int key[kK];
#pragma unroll
  for (int u = 0; u < kK; ++u) key[u] = 64 * u + lane < n ? idx[64 * u + lane] : -1;
  const int e = i < n ? idx[i] : -1;
  const typename El<TYPE>::raw* src = x + (size_t)((i < n ? i : 0) / k) * d;
  Vec<TYPE, VN> v[kA];
#pragma unroll
  for (int u = 0; u < kA; ++u)
    if (64 * u < pieces) v[u] = vec_load<TYPE, VN>(src + piece_start<VN>(64 * u + lane < pieces ? 64 * u + lane : pieces - 1, d));
  for (int b = blockIdx.x * 64 * kWaves + tid; b <= E; b += gridDim.x * 64 * kWaves) {
    int below = 0;
#pragma unroll
    for (int u = 0; u < kK; ++u)
      for (int j = 0; j < 64 && 64 * u + j < n; ++j)
        below += (unsigned)__builtin_amdgcn_readlane(key[u], j) < (unsigned)b;   // -1 is below none
    offsets[b] = below;
  }
  if (i >= n) return;
  if (e < 0 || e >= E) {
    if (lane == 0) row_of[i] = -1;
    return;
  }
  int row = 0;
#pragma unroll
  for (int u = 0; u < kK; ++u)
    row += __popcll(__ballot((unsigned)key[u] < (unsigned)e || (key[u] == e && 64 * u + lane < i)));
  if (lane == 0) {
    row_of[i] = row;
    pair_ids[row] = i;
  }
  typename El<TYPE>::raw* dst = out + (size_t)row * d;
  for (int c0 = 0; c0 < pieces; c0 += 64 * kA) {
#pragma unroll
    for (int u = 0; u < kA; ++u) {
      const int p = c0 + 64 * u + lane;
      if (c0 > 0 && p < pieces) v[u] = vec_load<TYPE, VN>(src + piece_start<VN>(p, d));
    }
#pragma unroll
    for (int u = 0; u < kA; ++u) {
      const int p = c0 + 64 * u + lane;
      if (p < pieces) vec_store<TYPE, VN>(dst + piece_start<VN>(p, d), v[u]);
    }
  }
}

// The whole sort in one launch, up to kWideMax pairs.  Each block places P
// consecutive pairs and copies their rows.  It counts all the keys for itself
// (LDS histogram; the low half of a counter takes every pair, the high half
// those before the block's own; WIDE, past 65535 pairs: two counters), scans the counts over the experts, ranks its
// pairs among themselves by ballots and adds the three.  The first row of each
// wave is on its way meanwhile, and a wave takes consecutive pairs: those of a
// token share one load, and a store waits for no load behind it (loads and
// stores return in order; rows strided over the waves took 46 us).
// 4096 tokens of 2048 bf16, ten pairs each: 42 us for 185 MB (4.4 TB/s), some
// 5 of it the count; histogram, scan, scatter and copy in four launches took 68.
constexpr int kOnePlaces = 256, kWidePlaces = 4096;     // pairs a block
constexpr int kOneMax = 65535, kWideMax = 256 * kWidePlaces;
constexpr int kOneThreads = 1024;
struct __attribute__((packed, aligned(4))) Key4 { int32_t v[4]; };

template <int TYPE, int VN, bool WIDE>
__global__ __launch_bounds__(kOneThreads) void sort_one_kernel(
    const typename El<TYPE>::raw* __restrict__ x, const int32_t* __restrict__ idx, int n, int k, int d, int E, int P,
    int32_t* __restrict__ offsets, int32_t* __restrict__ pair_ids, int32_t* __restrict__ row_of,
    typename El<TYPE>::raw* __restrict__ out) {
  constexpr int kA = 4;                         // pieces a lane holds ahead
  __shared__ uint32_t cnt[1024];                // counts, then the next free row of each expert
  __shared__ uint32_t earlier[WIDE ? 1024 : 1];
  __shared__ uint32_t wsum[16];
  __shared__ int place[WIDE ? kWidePlaces : kOnePlaces];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int first = blockIdx.x * P;
  const int mine = n - first < P ? n - first : P;
  const int pieces = (d + VN - 1) / VN;
  // a wave's pairs: consecutive ones, so that those of one token share a load
  const int per = (mine + kOneThreads / 64 - 1) / (kOneThreads / 64);
  const int q0 = wave * per, q1 = q0 + per < mine ? q0 + per : mine;
  Vec<TYPE, VN> ahead[kA];
  auto load = [&](int t, int c0) {
    const typename El<TYPE>::raw* src = x + (size_t)t * d;
#pragma unroll
    for (int u = 0; u < kA; ++u) {
      const int p = c0 + 64 * u + lane;
      if (c0 + 64 * u < pieces) ahead[u] = vec_load<TYPE, VN>(src + piece_start<VN>(p < pieces ? p : pieces - 1, d));
    }
  };
  if (q0 < q1) load((first + q0) / k, 0);
  if (tid < E) cnt[tid] = 0;
  if (WIDE && tid < E) earlier[tid] = 0;
  __syncthreads();
  auto count = [&](int j, int key) {
    if (key < 0 || key >= E) return;
    if (WIDE) {
      atomicAdd(&cnt[key], 1u);
      if (j < first) atomicAdd(&earlier[key], 1u);
    } else {
      atomicAdd(&cnt[key], j < first ? 0x10001u : 1u);
    }
  };
  constexpr int kQ = 4;                         // loads in flight
  const int quads = n >> 2;
  for (int q0 = tid; q0 < quads; q0 += kQ * kOneThreads) {
    Key4 v[kQ];
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      const int q = q0 + u * kOneThreads;
      v[u] = *reinterpret_cast<const Key4*>(idx + 4 * (q < quads ? q : q0));
    }
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      const int q = q0 + u * kOneThreads;
      if (q < quads) {
#pragma unroll
        for (int j = 0; j < 4; ++j) count(4 * q + j, v[u].v[j]);
      }
    }
  }
  if (tid < (n & 3)) count(4 * quads + tid, idx[4 * quads + tid]);
  int key = -1;
  if (wave == 0 && lane < mine) key = idx[first + lane];
  __syncthreads();
  const uint32_t both = tid < E ? cnt[tid] : 0;
  const uint32_t c = WIDE ? both : both & 0xFFFFu;
  const uint32_t own = WIDE ? (tid < E ? earlier[tid] : 0) : both >> 16;     // before the block's pairs
  const uint32_t incl = (uint32_t)wave_scan((int)c);
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int q = 0; q < kOneThreads / 64; ++q) before += q < wave ? wsum[q] : 0;
  if (tid < E) {
    const uint32_t lo = before + incl - c;
    cnt[tid] = lo + own;
    if (blockIdx.x == 0) {
      offsets[tid] = (int32_t)lo;
      if (tid == E - 1) offsets[E] = (int32_t)(before + incl);
    }
  }
  __syncthreads();
  if (wave == 0) {
    const int nb = 32 - __clz(E > 1 ? E - 1 : 1);
    for (int b0 = 0; b0 < mine; b0 += 64) {
      if (b0 > 0) key = b0 + lane < mine ? idx[first + b0 + lane] : -1;
      const bool valid = key >= 0 && key < E;
      uint64_t peers = __ballot(valid);
      for (int b = 0; b < nb; ++b) {
        const uint64_t on = __ballot((key >> b) & 1);
        peers &= ((key >> b) & 1) ? on : ~on;
      }
      const int rank = __popcll(peers & ((1ull << lane) - 1));
      int row = -1;
      if (valid) row = (int)cnt[key] + rank;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (valid && rank == 0) cnt[key] += (uint32_t)__popcll(peers);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (b0 + lane < mine) {
        place[b0 + lane] = row;
        row_of[first + b0 + lane] = row;
        if (valid) pair_ids[row] = first + b0 + lane;
      }
    }
  }
  __syncthreads();
  for (int c0 = 0; c0 < pieces; c0 += 64 * kA) {
    int held = c0 == 0 && q0 < q1 ? (first + q0) / k : -1;
    for (int q = q0; q < q1; ++q) {
      const int row = __builtin_amdgcn_readfirstlane(place[q]);
      const int t = (first + q) / k;
      if (row < 0) continue;
      if (t != held) load(held = t, c0);
      typename El<TYPE>::raw* dst = out + (size_t)row * d;
#pragma unroll
      for (int u = 0; u < kA; ++u) {
        const int p = c0 + 64 * u + lane;
        if (p < pieces) vec_store<TYPE, VN>(dst + piece_start<VN>(p, d), ahead[u]);
      }
    }
  }
}

// One wave per (token, PP x 64 pieces of its row): the rows of kB ranks in
// flight, summed in rank order.  WEIGHTED = false: the gradient of the sort
// (w = 1, no shared rows).  HBM-bound; each row is read once, so past the
// caches' replacement: 168 MB of rows, us: 38.2 with ordinary loads, 33.6 so,
// 31 so with PP = 4 (5.9 TB/s of a row's 4 KB in one wave).  Fewer tokens than
// kWideTokens take PP = 1, for more waves (64 tokens: 7.4 against 9.4).
constexpr int kWideTokens = 1024;
template <int TYPE, int VN, int PP, bool WEIGHTED>
__global__ __launch_bounds__(64 * kWaves) void unsort_kernel(
    const typename El<TYPE>::raw* __restrict__ rows, const int32_t* __restrict__ row_of, const float* __restrict__ w,
    const typename El<TYPE>::raw* __restrict__ shared, const float* __restrict__ sgate, int T, int k, int d,
    typename El<TYPE>::raw* __restrict__ y) {
  constexpr int kB = PP == 1 ? 10 : 4;
  const int lane = threadIdx.x & 63;
  const int pieces = (d + VN - 1) / VN;
  const unsigned slabs = (unsigned)(pieces + 64 * PP - 1) / (64 * PP);
  const long n = (long)T * k;
  for (unsigned item = (unsigned)wave_id(); item < (unsigned)T * slabs; item += (unsigned)wave_count()) {
    const int t = (int)(item / slabs);
    const int c0 = (int)(item % slabs) * 64 * PP + lane;
    int e[PP];
    bool mine[PP];
#pragma unroll
    for (int p = 0; p < PP; ++p) {
      mine[p] = c0 + 64 * p < pieces;
      e[p] = piece_start<VN>(mine[p] ? c0 + 64 * p : pieces - 1, d);
    }
    float acc[PP][VN];
#pragma unroll
    for (int p = 0; p < PP; ++p)
#pragma unroll
      for (int j = 0; j < VN; ++j) acc[p][j] = 0.f;
    for (int r0 = 0; r0 < k; r0 += kB) {
      Vec<TYPE, VN> v[kB][PP];
      float wv[kB];
      bool has[kB];
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        const long i = (long)t * k + (r0 + u < k ? r0 + u : k - 1);
        const int row = row_of[i];
        has[u] = r0 + u < k && row >= 0 && row < n;
        wv[u] = WEIGHTED ? w[i] : 1.f;
        const typename El<TYPE>::raw* src = rows + (size_t)(has[u] ? row : 0) * d;
#pragma unroll
        for (int p = 0; p < PP; ++p) v[u][p] = vec_load<TYPE, VN, true>(src + e[p]);
      }
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        if (has[u]) {
#pragma unroll
          for (int p = 0; p < PP; ++p)
#pragma unroll
            for (int j = 0; j < VN; ++j)
              acc[p][j] = WEIGHTED ? fmaf(wv[u], El<TYPE>::up(v[u][p].e[j]), acc[p][j])
                                   : acc[p][j] + El<TYPE>::up(v[u][p].e[j]);
        }
      }
    }
#pragma unroll
    for (int p = 0; p < PP; ++p) {
      if (WEIGHTED && shared) {
        const float s = sgate[t];
        const Vec<TYPE, VN> v = vec_load<TYPE, VN, true>(shared + (size_t)t * d + e[p]);
#pragma unroll
        for (int j = 0; j < VN; ++j) acc[p][j] = fmaf(s, El<TYPE>::up(v.e[j]), acc[p][j]);
      }
      Vec<TYPE, VN> o;
#pragma unroll
      for (int j = 0; j < VN; ++j) o.e[j] = El<TYPE>::down(acc[p][j]);
      if (mine[p]) vec_store<TYPE, VN>(y + (size_t)t * d + e[p], o);
    }
  }
}

// One wave per (token, rank), and one more a token for the shared rows: reads
// dy[t] (from L2 for all ranks but one) and its row, writes the row's gradient
// and their dot product.  HBM-bound: 390 MB in 79 us (4.9 TB/s).
template <int TYPE, int VN>
__global__ __launch_bounds__(64 * kWaves) void unsort_grad_kernel(
    const typename El<TYPE>::raw* __restrict__ dy, const typename El<TYPE>::raw* __restrict__ rows,
    const int32_t* __restrict__ row_of, const float* __restrict__ w, const typename El<TYPE>::raw* __restrict__ shared,
    const float* __restrict__ sgate, int T, int k, int d, typename El<TYPE>::raw* __restrict__ drows,
    float* __restrict__ dw, typename El<TYPE>::raw* __restrict__ dshared, float* __restrict__ dsgate) {
  constexpr int kB = 4;
  const int lane = threadIdx.x & 63;
  const int pieces = (d + VN - 1) / VN;
  const int per = k + (shared ? 1 : 0);
  const long n = (long)T * k;
  for (unsigned item = (unsigned)wave_id(); item < (unsigned)T * (unsigned)per; item += (unsigned)wave_count()) {
    const int t = (int)(item / (unsigned)per);
    const int r = (int)(item % (unsigned)per);
    const long i = (long)t * k + r;
    const typename El<TYPE>::raw* src;
    typename El<TYPE>::raw* dst;
    float f;
    if (r < k) {
      const int row = row_of[i];
      if (row < 0 || row >= n) {
        if (lane == 0) dw[i] = 0.f;
        continue;
      }
      src = rows + (size_t)row * d;
      dst = drows + (size_t)row * d;
      f = w[i];
    } else {
      src = shared + (size_t)t * d;
      dst = dshared + (size_t)t * d;
      f = sgate[t];
    }
    const typename El<TYPE>::raw* g = dy + (size_t)t * d;
    float dot = 0.f;
    for (int c0 = lane; c0 < pieces; c0 += 64 * kB) {
      Vec<TYPE, VN> a[kB], b[kB];
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        const int e = piece_start<VN>(c0 + 64 * u < pieces ? c0 + 64 * u : pieces - 1, d);
        a[u] = vec_load<TYPE, VN>(g + e);
        b[u] = vec_load<TYPE, VN, true>(src + e);
      }
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        const int c = c0 + 64 * u;
        if (c < pieces) {
          const int e = piece_start<VN>(c, d);
          const int again = c * VN - e;               // elements counted by the piece before
          Vec<TYPE, VN> o;
#pragma unroll
          for (int j = 0; j < VN; ++j) {
            const float gv = El<TYPE>::up(a[u].e[j]);
            o.e[j] = El<TYPE>::down(f * gv);
            dot = j >= again ? fmaf(gv, El<TYPE>::up(b[u].e[j]), dot) : dot;
          }
          vec_store<TYPE, VN>(dst + e, o);
        }
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) {
      if (r < k)
        dw[i] = dot;
      else
        dsgate[t] = dot;
    }
  }
}

// body(type tag, piece size tag) for a run-time element type and row length.
template <int V> struct Int { static constexpr int v = V; };
template <class F> int by_type(int type, int d, F&& body) {
  switch (type) {
    case MOE_TYPE_F32: return d >= 4 ? body(Int<MOE_TYPE_F32>{}, Int<4>{}) : body(Int<MOE_TYPE_F32>{}, Int<1>{});
    case MOE_TYPE_BF16: return d >= 8 ? body(Int<MOE_TYPE_BF16>{}, Int<8>{}) : body(Int<MOE_TYPE_BF16>{}, Int<1>{});
    case MOE_TYPE_F16: return d >= 8 ? body(Int<MOE_TYPE_F16>{}, Int<8>{}) : body(Int<MOE_TYPE_F16>{}, Int<1>{});
  }
  return MOE_ERR_INVALID_ARG;
}

struct SortWs {
  int32_t* counts;
  void* bucket;
  size_t bucket_bytes;
};
bool carve_sort(Carver& c, int T, int k, int E, SortWs* w) {
  w->counts = c.take<int32_t>(E);
  w->bucket_bytes = bucket_ws_bytes(T, k, E);
  w->bucket = c.take<uint8_t>(w->bucket_bytes);
  return c.ok();
}

__global__ void zero_i32_kernel(int32_t* p, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0;
}

// Sizes every entry point of this file takes.
int check_rows(int type, int T, int k, int d) {
  MOE_CHECK(type_size(type) != 0 && T >= 0 && k >= 1 && d >= 1);
  if (k > 1024 || d > (1 << 20) || (long)T * k > (1L << 30) || (long)T * (k + 1) > kMaxItems) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_sort_workspace_bytes(int32_t T, int32_t k, int32_t E) {
  if (T < 0 || k < 1 || k > 1024 || E < 1 || E > 1024 || (long)T * k > (1L << 30)) return 0;
  Carver c(nullptr, (size_t)-1);
  SortWs w;
  carve_sort(c, T, k, E, &w);
  return c.off + 256;
}

extern "C" int moe_sort_tokens(const void* x, int32_t type, int32_t T, int32_t d, const int32_t* idx, int32_t k,
                               int32_t E, void* x_sorted, int32_t* offsets, int32_t* pair_ids, int32_t* row_of,
                               void* ws, size_t ws_bytes, hipStream_t s) {
  MOE_TRY(check_rows(type, T, k, d));
  MOE_CHECK(E >= 1 && E <= 1024 && offsets);
  if (T == 0) {
    zero_i32_kernel<<<1, 256, 0, s>>>(offsets, E + 1);
    MOE_HIP(hipGetLastError());
    return MOE_OK;
  }
  const int es = type_size(type);
  MOE_CHECK(x && idx && x_sorted && pair_ids && row_of && ws);
  MOE_CHECK(aligned(x, es) && aligned(x_sorted, es) && aligned(ws, 256));
  MOE_CHECK(aligned(idx, 4) && aligned(offsets, 4) && aligned(pair_ids, 4) && aligned(row_of, 4));
  const long n = (long)T * k;
  Carver c(ws, ws_bytes);
  SortWs w;
  if (!carve_sort(c, T, k, E, &w)) return MOE_ERR_INVALID_ARG;
  if (n <= kFewMax)
    return by_type(type, d, [&](auto ty, auto vn) -> int {
      typedef typename El<decltype(ty)::v>::raw raw;
      sort_few_kernel<decltype(ty)::v, decltype(vn)::v><<<wave_grid(n), 64 * kWaves, 0, s>>>(
          static_cast<const raw*>(x), idx, (int)n, k, d, E, offsets, pair_ids, row_of, static_cast<raw*>(x_sorted));
      MOE_HIP(hipGetLastError());
      return MOE_OK;
    });
  // (few experts: the blocks' counters collide.  60000 pairs of one expert 65 us
  // in one launch, 25 in the four below; of eight 27 in both; 70000 of eight 43
  // and 27, of 512 25 and 71)
  if (n <= kWideMax && (n <= 8192 || E >= (n <= kOneMax ? 8 : 32))) {
    // pairs a block: a block for each of the 256 CUs, 16 pairs (one a wave) at least
    const int P = n <= 16 * 256 ? 16 : (int)((n + 255) / 256);
    return by_type(type, d, [&](auto ty, auto vn) -> int {
      typedef typename El<decltype(ty)::v>::raw raw;
      auto* kernel = n <= kOneMax ? sort_one_kernel<decltype(ty)::v, decltype(vn)::v, false>
                                  : sort_one_kernel<decltype(ty)::v, decltype(vn)::v, true>;
      kernel<<<(unsigned)((n + P - 1) / P), kOneThreads, 0, s>>>(static_cast<const raw*>(x), idx, (int)n, k, d, E, P,
                                                               offsets, pair_ids, row_of, static_cast<raw*>(x_sorted));
      MOE_HIP(hipGetLastError());
      return MOE_OK;
    });
  }
  MOE_TRY(bucket_launch(idx, T, k, E, w.counts, offsets, pair_ids, w.bucket, w.bucket_bytes, s, nullptr));
  return by_type(type, d, [&](auto ty, auto vn) -> int {
    typedef typename El<decltype(ty)::v>::raw raw;
    gather_rows_kernel<decltype(ty)::v, decltype(vn)::v><<<wave_grid(n), 64 * kWaves, 0, s>>>(
        static_cast<const raw*>(x), idx, n, k, d, E, offsets, pair_ids, row_of, static_cast<raw*>(x_sorted));
    MOE_HIP(hipGetLastError());
    return MOE_OK;
  });
}

namespace moe {
namespace {
template <bool WEIGHTED>
int unsort_launch(const void* rows, int type, int T, int k, int d, const int32_t* row_of, const float* w,
                  const void* shared, const float* sgate, void* y, hipStream_t s) {
  return by_type(type, d, [&](auto ty, auto vn) -> int {
    constexpr int VN = decltype(vn)::v;
    typedef typename El<decltype(ty)::v>::raw raw;
    constexpr int PP = VN == 1 ? 1 : 4;
    const long pieces = (d + VN - 1) / VN;
    const bool wide = PP > 1 && T >= kWideTokens && pieces > 128;
    const long items = T * ((pieces + (wide ? 64 * PP : 64) - 1) / (wide ? 64 * PP : 64));
    if (items > kMaxItems) return MOE_ERR_UNSUPPORTED;
    auto* kernel = wide ? unsort_kernel<decltype(ty)::v, VN, PP, WEIGHTED> : unsort_kernel<decltype(ty)::v, VN, 1, WEIGHTED>;
    kernel<<<wave_grid(items), 64 * kWaves, 0, s>>>(static_cast<const raw*>(rows), row_of, w,
                                                    static_cast<const raw*>(shared), sgate, T, k, d,
                                                    static_cast<raw*>(y));
    MOE_HIP(hipGetLastError());
    return MOE_OK;
  });
}
}  // namespace
}  // namespace moe

extern "C" int moe_sort_tokens_backward(const void* dx_sorted, int32_t type, int32_t T, int32_t k, int32_t d,
                                        const int32_t* row_of, void* dx, hipStream_t s) {
  MOE_TRY(check_rows(type, T, k, d));
  if (T == 0) return MOE_OK;
  const int es = type_size(type);
  MOE_CHECK(dx_sorted && row_of && dx);
  MOE_CHECK(aligned(dx_sorted, es) && aligned(dx, es) && aligned(row_of, 4));
  return unsort_launch<false>(dx_sorted, type, T, k, d, row_of, nullptr, nullptr, nullptr, dx, s);
}

extern "C" int moe_unsort_combine(const void* rows, int32_t type, int32_t T, int32_t k, int32_t d,
                                  const int32_t* row_of, const float* w, const void* shared, const float* sgate,
                                  void* y, hipStream_t s) {
  MOE_TRY(check_rows(type, T, k, d));
  if (T == 0) return MOE_OK;
  const int es = type_size(type);
  MOE_CHECK(rows && row_of && w && y);
  MOE_CHECK((shared == nullptr) == (sgate == nullptr));
  MOE_CHECK(aligned(rows, es) && aligned(y, es) && aligned(shared, es) && aligned(row_of, 4) && aligned(w, 4) &&
            aligned(sgate, 4));
  return unsort_launch<true>(rows, type, T, k, d, row_of, w, shared, sgate, y, s);
}

extern "C" int moe_unsort_combine_backward(const void* dy, const void* rows, int32_t type, int32_t T, int32_t k,
                                           int32_t d, const int32_t* row_of, const float* w, const void* shared,
                                           const float* sgate, void* drows, float* dw, void* dshared, float* dsgate,
                                           hipStream_t s) {
  MOE_TRY(check_rows(type, T, k, d));
  if (T == 0) return MOE_OK;
  const int es = type_size(type);
  MOE_CHECK(dy && rows && row_of && w && drows && dw);
  const bool has = shared != nullptr;
  MOE_CHECK((sgate != nullptr) == has && (dshared != nullptr) == has && (dsgate != nullptr) == has);
  MOE_CHECK(aligned(dy, es) && aligned(rows, es) && aligned(shared, es) && aligned(drows, es) && aligned(dshared, es));
  MOE_CHECK(aligned(row_of, 4) && aligned(w, 4) && aligned(sgate, 4) && aligned(dw, 4) && aligned(dsgate, 4));
  return by_type(type, d, [&](auto ty, auto vn) -> int {
    typedef typename El<decltype(ty)::v>::raw raw;
    const long waves = (long)T * (k + (has ? 1 : 0));
    unsort_grad_kernel<decltype(ty)::v, decltype(vn)::v><<<wave_grid(waves), 64 * kWaves, 0, s>>>(
        static_cast<const raw*>(dy), static_cast<const raw*>(rows), row_of, w, static_cast<const raw*>(shared), sgate,
        T, k, d, static_cast<raw*>(drows), dw, static_cast<raw*>(dshared), dsgate);
    MOE_HIP(hipGetLastError());
    return MOE_OK;
  });
}
