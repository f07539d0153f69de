// Products of 16-bit matrices in tiles: out[q][p] = sum_k Q[q][k] P[p][k] with
// fp32 sums on v_mfma_f32_32x32x16, for rows in expert order (a chunk of one
// expert's rows by a tile of its matrix) and for the gradients of the matrices
// (a tile of one expert's matrix, k over its rows).
//
// An operand's tile is held in LDS in one of two forms, by what is contiguous
// in memory: k ("rows of k", read as fragments by 16-byte LDS reads), or q / p
// itself ("rows of q", k apart, read by ds_read_b64_tr_b16, which turns four
// rows of 16 elements into four k of each of 16 lanes).  So the products of the
// way forward (both k), of dx = dy W (k; p) and of dW = dy^T x (q; p) take the
// matrices as they lie in memory, none is transposed first.
//
// Pieces of 16 bytes are XOR-swizzled within their row, so that a fragment's
// reads meet all banks evenly.
#pragma once

#include "chunks.h"
#include "elem.h"
#include "internal.h"

namespace moe {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_v __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_v __attribute__((ext_vector_type(8)));

template <int TYPE>
__device__ __forceinline__ f32x16_t mfma32(s16x8_t a, s16x8_t b, f32x16_t c) {
  if constexpr (TYPE == MOE_TYPE_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_v, a), __builtin_bit_cast(bf16x8_v, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_v, a), __builtin_bit_cast(f16x8_v, b), c, 0, 0, 0);
}

// v without its lowest `past` bits (a multiple of 16), zeros above.
__device__ __forceinline__ u32x4_t shift_down(u32x4_t v, int past) {
  const uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
  const uint64_t a = past == 0 ? lo : past < 64 ? lo >> past | hi << (64 - past) : past < 128 ? hi >> (past - 64) : 0;
  const uint64_t b = past < 64 ? hi >> past : 0;
  return (u32x4_t){(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
}
// Elements k .. k + 7 of a row of K, zeros past its end.  A piece over the end
// is the row's last 8 elements, shifted: loading it element by element means as
// many dependent waits (rows of 1001: 35 us for what takes 9).  Rows shorter
// than that have no other way.
__device__ __forceinline__ u32x4_t load_piece(const uint16_t* row, int k, int K) {
  if (K < 8) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (k + j < K) w[j / 2] |= (uint32_t)row[k + j] << (16 * (j & 1));
    return (u32x4_t){w[0], w[1], w[2], w[3]};
  }
  const int from = k < K - 8 ? k : K - 8;
  const u32x4_t v = *reinterpret_cast<const Piece16*>(row + from);
  return k == from ? v : shift_down(v, 16 * (k - from));
}

// s_waitcnt vmcnt <= N, lgkmcnt == 0, then s_barrier, and no memory access
// moved across it by the compiler.
template <int N> __device__ __forceinline__ void stage_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (0 << 8));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// LDS address of block-uniform p, hidden from the compiler: its alias tracking
// would wait for every DMA in flight before a read of LDS.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_void*)p);
}

// An operand of one block: R rows of q (or p), k in [0, K).
struct Operand {
  const uint8_t* base;          // KC: element (row 0, k 0); else (k 0, column 0)
  const uint8_t* base2;         // PAIR: the second matrix's
  const uint8_t* next;          // base in the second segment of k
  long ld;                      // elements from row to row (KC), from k to k (else)
  long col;                     // else: columns of the matrix before the first one
  int n;                        // rows (KC) or columns (else) that exist, of R
  int K;
};

constexpr uint32_t kNowhere = 0x80000000u;      // past the end of any buffer here
constexpr int kMaxLds = 160 << 10;              // of a block

// R rows of q by BK k of 16 bits: 2 R BK bytes, KC: [R][BK], else [BK][R].
// PAIR (KC): rows come from two matrices in turns of 32 (32 of the first, the
// same 32 of the second, ..).
template <bool KC, int R, int BK, int NT, bool PAIR>
struct Tile {
  static constexpr int kBytes = 2 * R * BK;
  static constexpr int kPieces = KC ? BK / 8 : R / 8;           // of a row
  static constexpr int kPer = kBytes / 16 / NT;                 // pieces a thread
  static_assert(kPer * NT * 16 == kBytes, "whole pieces a thread");

  // swizzle of a row's pieces
  static __device__ __forceinline__ int swz(int row) {
    if constexpr (KC)
      return BK == 128 ? row & 15 : BK == 64 ? (row & 7) ^ ((row >> 3) & 1) : (row >> 2) & 3;
    else
      // four rows' 64 bytes on four quarters of the 256 bytes of a pass
      return R == 64 ? 4 * ((row >> 1) & 1) : 4 * (row & 3);
  }
  static __device__ __forceinline__ int pos(int row, int piece) {
    return row * (16 * kPieces) + 16 * (piece ^ swz(row));
  }

  // Fragment of 32 rows of q from r0 and 16 k from 16 kk: lane l holds row
  // l % 32 and k 8 (l / 32) .. + 7.
  static __device__ __forceinline__ s16x8_t frag(const uint8_t* t, int r0, int kk, int lane) {
    if constexpr (KC) {
      return *reinterpret_cast<const s16x8_t*>(t + pos(r0 + (lane & 31), 2 * kk + (lane >> 5)));
    } else {
      typedef __attribute__((address_space(3))) s16x4_t lds4;
      // lane i of 16: row i / 4 of four, four columns i % 4 of 16; lanes 16..31 the next 16 columns
      const int i = lane & 15, row = 16 * kk + 8 * (lane >> 5) + (i >> 2);
      const int piece = r0 / 8 + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
      const int at = pos(row, piece) + 8 * (i & 1);             // rows 4 apart: the same swizzle
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(t + at));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(t + at + 4 * 16 * kPieces));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }

  // Row and piece of memory that go to the tile's 16 bytes number `at`.
  static __device__ __forceinline__ void source(int at, int* row, int* piece) {
    *row = at / kPieces;
    *piece = (at % kPieces) ^ swz(*row);
  }
  // PAIR: row r of the tile is row `m` of matrix r / 32 % 2
  static __device__ __forceinline__ int matrix_row(int row) { return PAIR ? (row >> 6) * 32 + (row & 31) : row; }

  // ---- sizes of whole 16-byte pieces: memory to LDS by the buffer unit
  uint32_t vo[kPer];
  __device__ __forceinline__ void plan(const Operand& o) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      int row, piece;
      source((int)(threadIdx.x >> 6) * (64 * kPer) + 64 * i + (threadIdx.x & 63), &row, &piece);
      if constexpr (KC)
        vo[i] = matrix_row(row) < o.n ? (uint32_t)(matrix_row(row) * o.ld * 2 + piece * 16) : kNowhere;
      else
        vo[i] = 8 * piece < o.n ? (uint32_t)(row * o.ld * 2 + piece * 16) : kNowhere;
    }
  }
  // k0 .. k0 + BK of the operand (all zeros where k0 >= K) to LDS address t.
  // A wave's turns are 1 KB apart; it starts at kWave bytes of the tile.
  static constexpr int kWave = 1024 * kPer;
  __device__ __forceinline__ void dma(const Operand& o, uint32_t t, int k0) const {
    const int left = o.K - k0;
    const uint32_t to = t + wave_uniform() * kWave;
    if constexpr (KC) {
      // PAIR: a wave's 32 rows are of one matrix
      static_assert(!PAIR || (kPieces == 8 && kPer == 4), "32 rows a wave");
      // (as arithmetic: of a choice of pointers the compiler makes a load from scratch memory)
      const uint8_t* b = o.base + (PAIR ? (o.base2 - o.base) & -(long)(wave_uniform() & 1) : 0);
      const rsrc_t r = make_rsrc(b + 2l * k0, left > 0 ? kNowhere - 1 : 0);
      if (left >= BK) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) dma16(r, to + 1024 * i, vo[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          int row, piece;
          source((int)(threadIdx.x >> 6) * (64 * kPer) + 64 * i + (threadIdx.x & 63), &row, &piece);
          dma16(r, to + 1024 * i, 8 * piece < left ? vo[i] : kNowhere);
        }
      }
    } else {
      const int rows = left < BK ? left : BK;   // of k
      const long bytes = 2 * ((rows - 1) * o.ld + ((o.n + 7) & ~7));
      const rsrc_t r = make_rsrc(o.base + 2l * k0 * o.ld, rows > 0 ? (uint32_t)bytes : 0);
#pragma unroll
      for (int i = 0; i < kPer; ++i) dma16(r, to + 1024 * i, vo[i]);
    }
  }
  static __device__ __forceinline__ int wave_uniform() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }
  static __device__ __forceinline__ void dma16(rsrc_t r, uint32_t to, uint32_t from) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(uintptr_t)to, 16, from, 0, 0, 0);
  }

  // ---- any size: through registers, vo as below.  Rows that do not exist are
  // the last one's, never stored; k past K are zeros.  Columns (not KC): a piece
  // over the last one is the matrix's last 8 columns, shifted by `past`.
  int past[KC ? 1 : kPer];
  __device__ __forceinline__ void plan_any(const Operand& o) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      int row, piece;
      source((int)threadIdx.x + NT * i, &row, &piece);
      if constexpr (KC) {
        const int r = matrix_row(row) < o.n ? matrix_row(row) : o.n - 1;
        vo[i] = (uint32_t)(r * o.ld * 2 + piece * 16);
      } else {
        // (columns from the matrix's first one: o.base is o.col before that)
        const int c = (int)o.col + 8 * piece, last = (int)o.col + o.n - 8, from = c < last || last < 0 ? c : last;
        vo[i] = (uint32_t)(row * o.ld * 2 + from * 2);
        past[i] = 16 * (c - from);
      }
    }
  }
  __device__ __forceinline__ void fetch(const Operand& o, int k0, u32x4_t (&v)[kPer]) const {
    if constexpr (KC) {
      const uint8_t* b1 = o.base + 2l * k0;
      const uint8_t* b2 = PAIR ? o.base2 + 2l * k0 : b1;
      if (k0 + BK <= o.K) {                     // whole pieces: one scalar base, one offset a piece
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = *reinterpret_cast<const Piece16*>(b1 + (second(i) ? b2 - b1 : 0) + vo[i]);
        return;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        int row, piece;
        source((int)threadIdx.x + NT * i, &row, &piece);
        const uint8_t* p = b1 + (second(i) ? b2 - b1 : 0) + (vo[i] - 16 * piece);
        v[i] = load_piece(reinterpret_cast<const uint16_t*>(p) - k0, k0 + 8 * piece, o.K);
      }
    } else {
      const uint8_t* b = o.base - 2 * o.col + 2l * k0 * o.ld;
      const bool wide = o.col + o.n >= 8;       // a matrix with 8 columns
      if (wide && k0 + BK <= o.K) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = *reinterpret_cast<const Piece16*>(b + vo[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          int row, piece;
          source((int)threadIdx.x + NT * i, &row, &piece);
          const bool in = k0 + row < o.K;
          const uint8_t* p = b + (in ? (long)vo[i] : (long)vo[i] - (long)(k0 + row - (o.K - 1)) * o.ld * 2);
          const u32x4_t w = wide ? (u32x4_t)*reinterpret_cast<const Piece16*>(p)
                                 : load_piece(reinterpret_cast<const uint16_t*>(p) - 8 * piece, 8 * piece, o.n);
          v[i] = in ? w : (u32x4_t){0, 0, 0, 0};
        }
      }
      if (wide && o.n < R) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = shift_down(v[i], past[i]);
      }
    }
  }
  // PAIR: whether a thread's piece i is of the second matrix (the same for its wave)
  static __device__ __forceinline__ bool second(int i) {
    if constexpr (!PAIR) return false;
    if constexpr (NT / kPieces == 32) return i & 1;             // 32 rows a turn of the block
    return __builtin_amdgcn_readfirstlane(((int)threadIdx.x + NT * i) / kPieces) & 32;
  }
  __device__ __forceinline__ void put(uint8_t* t, const u32x4_t (&v)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) *reinterpret_cast<u32x4_t*>(t + 16 * ((int)threadIdx.x + NT * i)) = v[i];
  }
};

// Block shape: WQ x WP waves of TQ x TP tiles of 32 x 32, k in steps of BK
// through NS stages.  AL: rows are whole 16-byte pieces at 16-byte addresses.
template <int TYPE_, bool QK_, bool PK_, int WQ_, int WP_, int TQ_, int TP_, int BK_, int NS_, bool PAIR_, bool AL_, int WAVES_ = 1>
struct Shape {
  static constexpr int TYPE = TYPE_, WQ = WQ_, WP = WP_, TQ = TQ_, TP = TP_, BK = BK_, NS = AL_ ? NS_ : 2;
  static constexpr int WAVES = WAVES_;           // a SIMD at least
  static constexpr bool QK = QK_, PK = PK_, PAIR = PAIR_, AL = AL_;
  static constexpr int NT = 64 * WQ * WP, BQ = 32 * WQ * TQ, BP = 32 * WP * TP;
  static constexpr int AHEAD = TQ * TP >= 4 ? 1 : PAIR ? 4 : 6;            // !AL: steps in registers
  typedef Tile<QK, BQ, BK, NT, false> QT;
  typedef Tile<PK, BP, BK, NT, PAIR> PT;
  static constexpr int kStage = QT::kBytes + PT::kBytes;
  static constexpr int kStages = NS * kStage;
};

// acc[q][p] += the products of one step of k, for the first LIVE of the wave's
// tiles of q (LIVE is a constant: with a branch around each tile every
// fragment's read is waited for before its products).  Fragments are read while
// the products of the 16 k before run.
template <class S, int LIVE>
__device__ __forceinline__ void tile_step(const uint8_t* st, int lane, int wq, int wp, f32x16_t (&acc)[S::TQ][S::TP]) {
  if constexpr (LIVE > 0) {
    s16x8_t p[2][S::TP], q[2][LIVE];
    const auto read = [&](int kk) {
#pragma unroll
      for (int t = 0; t < S::TP; ++t) p[kk & 1][t] = S::PT::frag(st + S::QT::kBytes, 32 * (wp * S::TP + t), kk, lane);
#pragma unroll
      for (int t = 0; t < LIVE; ++t) q[kk & 1][t] = S::QT::frag(st, 32 * (wq * S::TQ + t), kk, lane);
    };
    read(0);
#pragma unroll
    for (int kk = 0; kk < S::BK / 16; ++kk) {
      if (kk + 1 < S::BK / 16) read(kk + 1);
#pragma unroll
      for (int u = 0; u < LIVE; ++u)
#pragma unroll
        for (int t = 0; t < S::TP; ++t) acc[u][t] = mfma32<S::TYPE>(p[kk & 1][t], q[kk & 1][u], acc[u][t]);
    }
    constexpr int kFirst = (S::PK ? 1 : 2) * S::TP + (S::QK ? 1 : 2) * LIVE;    // LDS reads of a kk
    __builtin_amdgcn_sched_group_barrier(0x100, kFirst, 0);
#pragma unroll
    for (int kk = 0; kk < S::BK / 16; ++kk)
#pragma unroll
      for (int m = 0; m < LIVE * S::TP; ++m) {
        if (kk + 1 < S::BK / 16) {              // reads spread over the products
          constexpr int kEach = kFirst / (LIVE * S::TP), kMore = kFirst % (LIVE * S::TP);
          if (m < kMore)
            __builtin_amdgcn_sched_group_barrier(0x100, kEach + 1, 0);
          else if (kEach > 0)
            __builtin_amdgcn_sched_group_barrier(0x100, kEach, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
  }
}

// acc[q][p] += the product over k, in one segment or two of K each (of the
// operands at base, then at next).
template <class S, int SEGS, int LIVE>
__device__ __forceinline__ void tile_loop(Operand qo, Operand po, uint8_t* lds, f32x16_t (&acc)[S::TQ][S::TP]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wq = wave / S::WP, wp = wave % S::WP;
  const int per = (qo.K + S::BK - 1) / S::BK, steps = SEGS * per;
  typename S::QT qt;
  typename S::PT pt;
  if constexpr (S::AL) {
    constexpr int kDma = S::QT::kPer + S::PT::kPer;
    qt.plan(qo);
    pt.plan(po);
    const uint32_t base = lds_address(lds);
    const auto issue = [&](int s, uint32_t st) {
      if (SEGS == 2 && s == per) {
        qo.base = qo.next;
        po.base = po.next;
      }
      const int k0 = s < steps ? (SEGS == 2 && s >= per ? s - per : s) * S::BK : qo.K;
      qt.dma(qo, base + st, k0);
      pt.dma(po, base + st + S::QT::kBytes, k0);
    };
#pragma unroll
    for (int s = 0; s < S::NS - 1; ++s) issue(s, s * S::kStage);
    uint32_t now = 0, fill = (S::NS - 1) * S::kStage;           // stages, as bytes
    const auto after = [](uint32_t st) { return st == (S::NS - 1) * S::kStage ? 0 : st + S::kStage; };
    for (int s = 0; s < steps; ++s) {
      stage_wait<(S::NS - 2) * kDma>();
      issue(s + S::NS - 1, fill);
      tile_step<S, LIVE>(lds + now, lane, wq, wp, acc);
      now = after(now);
      fill = after(fill);
    }
    stage_wait<0>();
  } else {
    // AHEAD steps in registers, then LDS
    constexpr int D = S::AHEAD;
    u32x4_t qv[D][S::QT::kPer], pv[D][S::PT::kPer];
    qt.plan_any(qo);
    pt.plan_any(po);
    const auto fetch = [&](int s, int d) {
      const bool second = SEGS == 2 && s >= per;
      Operand q = qo, p = po;
      if (second) {
        q.base = qo.next;
        p.base = po.next;
      }
      const int k0 = (second ? s - per : s) * S::BK;
      qt.fetch(q, k0, qv[d]);
      pt.fetch(p, k0, pv[d]);
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (d < steps) fetch(d, d);
    for (int s = 0; s < steps; s += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (s + d >= steps) break;
        // the other buffer is read in the step before: one barrier a step
        uint8_t* st = lds + ((s + d) & 1) * S::kStage;
        qt.put(st, qv[d]);
        pt.put(st + S::QT::kBytes, pv[d]);
        if (s + d + D < steps) fetch(s + d + D, d);
        stage_wait<63>();
        tile_step<S, LIVE>(st, lane, wq, wp, acc);
      }
    }
    stage_wait<63>();
  }
}

template <class S, int SEGS>
__device__ __forceinline__ void tile_product(const Operand& q, const Operand& p, uint8_t* lds, int live,
                                             f32x16_t (&acc)[S::TQ][S::TP]) {
  // every wave meets the same barriers, whichever loop it is in
  if (live == S::TQ) return tile_loop<S, SEGS, S::TQ>(q, p, lds, acc);
  if constexpr (S::TQ > 3)
    if (live == 3) return tile_loop<S, SEGS, 3>(q, p, lds, acc);
  if constexpr (S::TQ > 2)
    if (live == 2) return tile_loop<S, SEGS, 2>(q, p, lds, acc);
  if constexpr (S::TQ > 1)
    if (live == 1) return tile_loop<S, SEGS, 1>(q, p, lds, acc);
  tile_loop<S, SEGS, 0>(q, p, lds, acc);
}

// LDS of a wave that turns 32 rows of 32 NP columns (store_rows), each padded by
// a piece.
template <int OUT, int NP> constexpr int kTurn = 32 * (32 * NP * (int)sizeof(typename El<OUT>::raw) + 16);
// LDS of a block: its stages, then in their place the turns of its waves, which
// may need more (fp32 in tiles of 128 x 128 in half steps: 34 KB, stages 32; three
// blocks a CU all the same).
template <class S, int OUT>
constexpr int kBlockLds = S::kStages > S::NT / 64 * kTurn<OUT, S::TP> ? S::kStages : S::NT / 64 * kTurn<OUT, S::TP>;

// 32 rows of q by 32 NP columns of p, one wave: from the sums' layout (lane:
// row l % 32, columns 8 (i / 4) + 4 (l / 32) + i % 4 of each 32) through the
// wave's own LDS to rows in memory, each rounded once to OUT.  out: (row 0,
// column 0); rows and cols that exist; rows whole 16-byte pieces (AL) or not.
// Stores past the caches, which keep what the other blocks read (a training
// step's calls on 4096 x 8 rows of 256 experts 1840 -> 1779 us in all).
template <int OUT, int NP, bool AL>
__device__ __forceinline__ void store_rows(uint8_t* lds, const f32x16_t* v, void* out, long ld, int rows, int cols) {
  typedef typename El<OUT>::raw raw;
  constexpr int kN = El<OUT>::kN;               // elements of a piece
  constexpr int kPitch = kTurn<OUT, NP> / 32;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int t = 0; t < NP; ++t)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      typedef raw raw4 __attribute__((ext_vector_type(4)));
      raw4 e;
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = El<OUT>::down(v[t][4 * b + i]);
      *reinterpret_cast<raw4*>(lds + (lane & 31) * kPitch + (32 * t + 8 * b + 4 * (lane >> 5)) * sizeof(raw)) = e;
    }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  constexpr int kRow = 32 * NP / kN;            // pieces a row
#pragma unroll
  for (int j = 0; j < 32 * kRow / 64; ++j) {
    const int at = 64 * j + lane, row = at / kRow, c = (at % kRow) * kN;
    if (row < rows && c < cols) {
      const uint8_t* from = lds + row * kPitch + c * sizeof(raw);
      raw* to = reinterpret_cast<raw*>(out) + row * ld + c;
      if (AL || c + kN <= cols) {
        __builtin_nontemporal_store(*reinterpret_cast<const u32x4_t*>(from), reinterpret_cast<Piece16*>(to));
      } else {
        for (int i = 0; c + i < cols; ++i) to[i] = reinterpret_cast<const raw*>(from)[i];
      }
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Which (unit, tile) a block works on.  Workgroups go to the 8 XCDs in turn,
// each with its own L2: an XCD takes whole groups of `group` neighbouring units
// (chunks of rows, or tiles of q) with all their tiles of p, so that what the
// tiles share is read into one L2 (by_unit); or, where units are few, a range
// of the tiles of p for all units.
struct Grid {
  int by_unit, group;
  int tiles;                    // of p
  int per_xcd;                  // !by_unit: tiles of p of an XCD
  int unit0, units;             // this launch's
};
__device__ __forceinline__ bool grid_place(const Grid& g, int* unit, int* tile) {
  const int xcd = blockIdx.x & 7, at = (int)(blockIdx.x >> 3);
  const int row = g.by_unit ? g.tiles : g.per_xcd;
  const int band = at / (g.group * row), in = at - band * (g.group * row);
  const int u = in % g.group, t = in / g.group;
  const int v = g.by_unit ? (band * 8 + xcd) * g.group + u : band * g.group + u;
  *unit = g.unit0 + v;
  *tile = g.by_unit ? t : xcd * g.per_xcd + t;
  return v < g.units && *tile < g.tiles;
}
constexpr long kMaxBlocks = 1l << 22;           // of a launch (its threads are counted in 32 bits)
// launch(grid, blocks) for all units, in as few launches as that allows
template <class F> int grid_launch(long units, long tiles, int group, F launch) {
  Grid g{};
  g.tiles = (int)tiles;
  g.group = group;
  g.per_xcd = (int)((tiles + 7) / 8);
  const long row = 8l * g.per_xcd;              // blocks a unit, at most
  const long per = kMaxBlocks / row / (8 * group) * (8 * group);
  if (per < 1) return MOE_ERR_UNSUPPORTED;
  for (long u = 0; u < units; u += per) {
    g.unit0 = (int)u;
    g.units = (int)(units - u < per ? units - u : per);
    g.by_unit = g.units >= 16 * group;
    const long bands = g.by_unit ? (g.units + 8 * group - 1) / (8 * group) : (g.units + group - 1) / group;
    MOE_TRY(launch(g, (unsigned)(8 * bands * group * (g.by_unit ? tiles : g.per_xcd))));
  }
  return MOE_OK;
}

// Block shapes.  Large: 128 x 128, two blocks a CU, so that one's products fill
// the other's waits.  Wide: 256 x 256 by 8 waves of 128 x 64, which read a third
// less from LDS for a product and leave one block a CU.  Small: 64 x 64 (PAIR 64
// x 128), where larger ones would leave CUs idle; there a step's fixed cost
// counts (barrier, loads issued, first fragments: about 0.35 us against 0.06 of
// products), so steps are twice as long where the columns of P are turned (256 x
// 4096 dx 51 -> 35 us; forward 22 -> 28, which keeps five stages).
// Mats (gradients of matrices, few steps of k a tile): 128 x 128 in half steps,
// three blocks a CU (dW of 32768 rows of 256 experts, 2 x 512 x 2048: 388 us, 424
// as Large; 512 x 2048 184 and 213).
template <int TYPE, bool QK, bool PK, bool PAIR, bool AL>
using Large = Shape<TYPE, QK, PK, 2, 2, 2, 2, 64, 2, PAIR, AL, 2>;
template <int TYPE, bool QK, bool PK, bool PAIR>
using Wide = Shape<TYPE, QK, PK, 2, 4, 4, 2, 64, 2, PAIR, true, 2>;
template <int TYPE, bool QK, bool PK, bool PAIR, bool AL>
using Small = Shape<TYPE, QK, PK, 2, 2, 1, PAIR ? 2 : 1, PK || !AL ? 64 : 128, PAIR ? 4 : PK ? 5 : 2, PAIR, AL, 2>;
template <int TYPE, bool AL>
using Mats = Shape<TYPE, false, false, 2, 2, 2, 2, 32, 2, false, AL, AL ? 3 : 2>;

// ------------------------------------------------- rows of x by a matrix
struct RowsArgs {
  const uint8_t* q;             // rows [N][q_ld]
  long q_ld;
  const uint8_t *p, *p2;        // the experts' matrices; the second ones (PAIR, or the second segment of k)
  uint64_t p_stride, p2_stride; // bytes from expert to expert
  long p_ld;
  int K, P;                     // k of a segment; columns of the output
  const int32_t* offsets;       // [E + 1], or null: one matrix for all rows
  int E;
  long N;
  int act;
  void* out;                    // [N][P]
  float* pre;                   // null, or [N][2 P]
  Grid grid;
};

__device__ __forceinline__ float sigmoid_fast(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}
constexpr float kGeluB = 1.5957691216057308f;   // 2 sqrt(2 / pi): gelu_tanh(g) = g sigmoid(kGeluB (g + 0.044715 g^3))
// Phi(g), the normal distribution, and e = exp(-g^2 / 2).  With z = |g| / sqrt 2
// and t = 1 / (1 + 0.45 z), erfc(z) exp(z^2) / (2 t) is smooth on 0 < t <= 1: a
// polynomial of degree 9 fitted to it (least largest relative error, 3.2e-8).
// The tail keeps its relative precision, which 1 + erf would lose (and the
// library's erfc took 10 us of 59 for 4200 rows of 1001 x 2 x 347).
__device__ __forceinline__ float normal(float g, float* e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.45f * 0.70710678118654752f, fabsf(g), 1.f));
  constexpr float c[10] = {1.269426604e-01f, 1.269415815e-01f, 1.141358193e-01f, 8.762608203e-02f, 5.997511320e-02f,
                           -1.117864780e-02f, 7.119989770e-02f, -1.502906264e-01f, 9.534360267e-02f, -2.069547559e-02f};
  float q = c[9];
#pragma unroll
  for (int i = 8; i >= 0; --i) q = fmaf(q, t, c[i]);
  *e = __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f);
  const float tail = q * t * *e;
  return g < 0.f ? tail : 1.f - tail;
}
__device__ __forceinline__ float act_value(int act, float g) {
  float e;
  if (act == MOE_ACT_SILU) return g * sigmoid_fast(g);
  if (act == MOE_ACT_GELU) return g * normal(g, &e);
  return g * sigmoid_fast(kGeluB * (g + 0.044715f * g * g * g));
}
// act(g) and its derivative
__device__ __forceinline__ float act_slope(int act, float g, float* value) {
  if (act == MOE_ACT_GELU) {
    float e;
    const float p = normal(g, &e);
    *value = g * p;
    return fmaf(g, 0.39894228040143268f * e, p);
  }
  const bool silu = act == MOE_ACT_SILU;
  const float s = sigmoid_fast(silu ? g : kGeluB * (g + 0.044715f * g * g * g));
  *value = g * s;
  if (fabsf(g) > 1e4f) return s;                // s is 0 or 1 here, and g * g might overflow
  return s * fmaf(g * (1.f - s), silu ? 1.f : kGeluB * fmaf(0.134145f * g, g, 1.f), 1.f);
}

// A block: a chunk of rows by a tile of columns.  GATED: out = act(x p^T)
// (x p2^T), and both products before it to pre.
// Measured: 4096 rows, 2048 -> 2 x 8192 with pre 287 us (960 TFLOP/s, a library
// product of 8192 reaches 1455), its dx 363 (757: 512 tiles of 128 x 128 in one
// round, 128 of 256 x 256 would fill half the CUs); 8192 x 8192 -> 8192 886 us
// (1240), with fp32 y 902.  Bound by the matrix cores waiting for each step's barrier and first
// fragments.  32768 rows of 256 experts, 2048 -> 2 x 512 with pre 281 us, dx 298
// (4.9 and 4.3 TB/s of what they have to move): by HBM, and by buckets that fill
// three quarters of their chunks.
template <class S, int SEGS, bool GATED, int OUT>
__global__ __launch_bounds__(S::NT, S::WAVES) void rows_kernel(RowsArgs a) {
  extern __shared__ uint8_t tile_lds[];
  static_assert(!GATED || (S::PAIR && S::TP % 2 == 0), "tiles of both matrices in a wave");
  static_assert(S::NT / 64 * kTurn<OUT, S::TP> <= kBlockLds<S, OUT> && kBlockLds<S, OUT> <= kMaxLds, "turns in LDS");
  static_assert(!GATED || kTurn<MOE_TYPE_F32, S::TP / 2> <= kTurn<OUT, S::TP>, "saved products turned in the same place");
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
  constexpr int kCols = GATED ? S::BP / 2 : S::BP;
  const int p0 = tile * kCols;
  const int cols = a.P - p0 < kCols ? a.P - p0 : kCols;
  Operand q{}, p{};
  q.base = a.q + 2 * start * a.q_ld;
  q.next = q.base + 2l * a.K;
  q.ld = a.q_ld;
  q.n = n;
  q.K = p.K = a.K;
  const uint64_t off = 2ull * (uint64_t)p0 * (S::PK ? a.p_ld : 1);
  p.base = a.p + (uint64_t)e * a.p_stride + off;
  p.base2 = p.next = a.p2 + (uint64_t)e * a.p2_stride + off;
  p.ld = a.p_ld;
  p.col = p0;
  p.n = cols;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wq = wave / S::WP, wp = wave % S::WP;
  const int left = n - 32 * wq * S::TQ;
  const int live = left <= 0 ? 0 : left >= 32 * S::TQ ? S::TQ : (left + 31) / 32;
  f32x16_t acc[S::TQ][S::TP] = {};
  tile_product<S, SEGS>(q, p, tile_lds, live, acc);
  uint8_t* mine = tile_lds + wave * kTurn<OUT, S::TP>;
#pragma unroll
  for (int t = 0; t < S::TQ; ++t) {
    if (t >= live) continue;
    const long r0 = start + 32 * (wq * S::TQ + t);
    const int rows = left - 32 * t < 32 ? left - 32 * t : 32;
    if constexpr (GATED) {
      constexpr int kH = S::TP / 2;
      const int c0 = 32 * kH * wp, have = cols - c0;
      f32x16_t h[kH], g[kH], u[kH];
#pragma unroll
      for (int j = 0; j < kH; ++j) {
        g[j] = acc[t][2 * j];
        u[j] = acc[t][2 * j + 1];
#pragma unroll
        for (int i = 0; i < 16; ++i) h[j][i] = act_value(a.act, g[j][i]) * u[j][i];
      }
      store_rows<OUT, kH, S::AL>(mine, h, static_cast<uint8_t*>(a.out) + kSize * (r0 * a.P + p0 + c0), a.P, rows, have);
      if (a.pre) {
        float* to = a.pre + 2 * r0 * a.P + p0 + c0;
        store_rows<MOE_TYPE_F32, kH, S::AL>(mine, g, to, 2l * a.P, rows, have);
        store_rows<MOE_TYPE_F32, kH, S::AL>(mine, u, to + a.P, 2l * a.P, rows, have);
      }
    } else {
      const int c0 = 32 * S::TP * wp;
      store_rows<OUT, S::TP, S::AL>(mine, acc[t], static_cast<uint8_t*>(a.out) + kSize * (r0 * a.P + p0 + c0), a.P, rows,
                                    cols - c0);
    }
  }
}

// ------------------------------------------- gradients of the matrices
struct MatsArgs {
  const uint8_t *q, *p;         // [N][q_ld], [N][p_ld]
  long q_ld, p_ld;
  int Q, P;                     // the matrix: dW[Q][P] = sum over an expert's rows of q p
  int q_tiles;                  // of a matrix
  int mats;                     // 1, or 2: columns Q .. 2 Q - 1 of q give the second matrix
  const int32_t* offsets;
  int E;
  long N;
  void *out, *out2;
  uint64_t out_stride, out2_stride;             // bytes from expert to expert
  Grid grid;
};
// A block's expert and tile of q, with its columns of p from p0.
struct MatsTile {
  Operand q, p;
  int q0;
  uint8_t* out;                 // the matrix
};
template <class S> __device__ __forceinline__ MatsTile mats_tile(const MatsArgs& a, int unit, int p0) {
  const int per = a.mats * a.q_tiles, e = unit / per, qt = unit - e * per;
  const int second = qt >= a.q_tiles ? 1 : 0;
  long start = 0, end = a.N;
  if (a.offsets) {
    start = row_border(a.offsets[e], (int)a.N);
    end = row_border(a.offsets[e + 1], (int)a.N);
    if (end < start) end = start;
  }
  MatsTile m{};
  m.q0 = (qt - second * a.q_tiles) * S::BQ;
  m.q.base = a.q + 2 * (start * a.q_ld + second * a.Q + m.q0);
  m.q.ld = a.q_ld;
  m.q.col = second * a.Q + m.q0;
  m.q.n = a.Q - m.q0 < S::BQ ? a.Q - m.q0 : S::BQ;
  m.p.base = a.p + 2 * (start * a.p_ld + p0);
  m.p.ld = a.p_ld;
  m.p.col = p0;
  m.p.n = a.P - p0 < S::BP ? a.P - p0 : S::BP;
  m.q.K = m.p.K = (int)(end - start);
  m.out = second ? static_cast<uint8_t*>(a.out2) + (uint64_t)e * a.out2_stride
                 : static_cast<uint8_t*>(a.out) + (uint64_t)e * a.out_stride;
  return m;
}
// A block: a tile of one expert's matrix, k over the expert's rows.
// Measured: 32768 rows of 256 experts, 2 x 512 x 2048 379 us (in fp32 500).
// Writing the 1.07 GB alone takes 172 (no rows), the products of 128 rows alone
// about 130 at the dense rate (4096 rows, 2 x 8192 x 2048: 257 us, 1070 TFLOP/s); the two overlap
// little, since a tile's loads, few steps and stores follow one another, at four
// blocks a CU as at one.
template <class S, int OUT>
__global__ __launch_bounds__(S::NT, S::WAVES) void mats_kernel(MatsArgs a) {
  extern __shared__ uint8_t tile_lds[];
  static_assert(S::NT / 64 * kTurn<OUT, S::TP> <= kBlockLds<S, OUT> && kBlockLds<S, OUT> <= kMaxLds, "turns in LDS");
  constexpr int kSize = El<OUT>::kN == 4 ? 4 : 2;
  int unit, tile;
  if (!grid_place(a.grid, &unit, &tile)) return;
  const int p0 = tile * S::BP;
  const MatsTile m = mats_tile<S>(a, unit, p0);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wq = wave / S::WP, wp = wave % S::WP;
  const int left = m.q.n - 32 * wq * S::TQ;
  const int live = left <= 0 ? 0 : left >= 32 * S::TQ ? S::TQ : (left + 31) / 32;
  f32x16_t acc[S::TQ][S::TP] = {};
  tile_product<S, 1>(m.q, m.p, tile_lds, live, acc);
  uint8_t* mine = tile_lds + wave * kTurn<OUT, S::TP>;
#pragma unroll
  for (int t = 0; t < S::TQ; ++t) {
    if (t >= live) continue;
    const long r0 = m.q0 + 32 * (wq * S::TQ + t);
    const int c0 = p0 + 32 * S::TP * wp;
    store_rows<OUT, S::TP, S::AL>(mine, acc[t], m.out + kSize * (r0 * a.P + c0), a.P,
                                  left - 32 * t < 32 ? left - 32 * t : 32, a.P - c0);
  }
}

}  // namespace moe
