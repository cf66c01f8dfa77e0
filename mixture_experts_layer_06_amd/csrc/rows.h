// rows.h — device helpers of the kernels that work along rows: vector access at
// any alignment, and sums and maxima over groups of lanes.
#pragma once

#include "common.h"

namespace moe {
namespace {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, bf16_t& o) { o = f32_to_bf16(v); }

// V elements of a row, starting anywhere: one wide access, which the hardware
// takes at the element's alignment.
template <typename T, int V>
struct __attribute__((packed, aligned(sizeof(T)))) Vec {
  T v[V];
};

// Elements j .. j+V-1 of a row of n; those past the end are zeros.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* __restrict__ row, int j, int n) {
  Vec<T, V> r;
  if (j + V <= n) {
    r = *reinterpret_cast<const Vec<T, V>*>(row + j);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = j + i < n ? row[j + i] : T(0);
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* __restrict__ row, int j, int n, const Vec<T, V>& x) {
  if (j + V <= n) {
    *reinterpret_cast<Vec<T, V>*>(row + j) = x;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (j + i < n) row[j + i] = x.v[i];
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

// f over aligned groups of L lanes (a power of two), the result in every lane of
// the group, the same in each: every step combines two disjoint halves, f being
// symmetric. Inside 16 lanes by DPP moves (a quad's pairs, its halves, then the
// mirrored half row and row), across them by gfx950's row and half-wave swaps.
template <int L, typename F>
__device__ __forceinline__ float over_lanes(float v, F f) {
  if (L > 1) v = f(v, dpp<0xB1>(v));   // quad_perm 1,0,3,2
  if (L > 2) v = f(v, dpp<0x4E>(v));   // quad_perm 2,3,0,1
  if (L > 4) v = f(v, dpp<0x141>(v));  // row_half_mirror
  if (L > 8) v = f(v, dpp<0x140>(v));  // row_mirror
  if (L > 16) {
    const u32x2_t s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(s.x), __uint_as_float(s.y));
  }
  if (L > 32) {
    const u32x2_t s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(s.x), __uint_as_float(s.y));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return over_lanes<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  return over_lanes<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace
}  // namespace moe
