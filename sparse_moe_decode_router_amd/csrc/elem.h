// Row elements in fp32, bf16 or fp16: pieces of up to 16 bytes moved between
// memory and fp32 registers.  Rows of odd length start at any element, so a
// piece is only element-aligned (gfx950 global loads and stores take such
// addresses).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe355.h"

namespace moe {

inline int type_size(int t) { return t == MOE_TYPE_F32 ? 4 : (t == MOE_TYPE_BF16 || t == MOE_TYPE_F16) ? 2 : 0; }

typedef uint32_t Piece16 __attribute__((ext_vector_type(4), aligned(2)));

// El<type>: kN elements of a 16-byte piece; rounding to nearest even, NaN kept.
template <int TYPE> struct El;
template <> struct El<MOE_TYPE_F32> {
  typedef float raw;
  static constexpr int kN = 4;
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float v) { return v; }
};
template <> struct El<MOE_TYPE_BF16> {
  typedef __bf16 raw;
  static constexpr int kN = 8;
  static __device__ __forceinline__ float up(__bf16 v) { return (float)v; }
  static __device__ __forceinline__ __bf16 down(float v) { return (__bf16)v; }
};
template <> struct El<MOE_TYPE_F16> {
  typedef _Float16 raw;
  static constexpr int kN = 8;
  static __device__ __forceinline__ float up(_Float16 v) { return (float)v; }
  static __device__ __forceinline__ _Float16 down(float v) { return (_Float16)v; }
};

// VN elements at p (VN = kN: one 16-byte access; VN = 1: one element).
template <int TYPE, int VN> struct Vec {
  typename El<TYPE>::raw e[VN];
};
// ONCE: read a single time (kept out of the way of what the caches hold).
template <int TYPE, int VN, bool ONCE = false>
__device__ __forceinline__ Vec<TYPE, VN> vec_load(const typename El<TYPE>::raw* p) {
  Vec<TYPE, VN> r;
  if constexpr (VN == 1) {
    r.e[0] = p[0];
  } else {
    const Piece16* q = reinterpret_cast<const Piece16*>(p);
    r = __builtin_bit_cast(Vec<TYPE, VN>, ONCE ? __builtin_nontemporal_load(q) : *q);
  }
  return r;
}
template <int TYPE, int VN>
__device__ __forceinline__ void vec_store(typename El<TYPE>::raw* p, const Vec<TYPE, VN>& v) {
  if constexpr (VN == 1)
    p[0] = v.e[0];
  else
    *reinterpret_cast<Piece16*>(p) = __builtin_bit_cast(Piece16, v);
}

}  // namespace moe
