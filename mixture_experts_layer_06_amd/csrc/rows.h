// rows.h — device helpers of the kernels that work along rows: vector access at
// any alignment, and sums and maxima over groups of lanes.
#pragma once

#include "block.h"

namespace moe {
namespace {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, bf16_t& o) { o = f32_to_bf16(v); }

// How the rows of a call lie, decided on the host by their length n:
//  kWhole   n is a multiple of the access and rows start on 16 bytes: an access is
//           inside the row or past it
//  kLoose   rows start anywhere (the hardware takes wide accesses at the element's
//           alignment) and have at least one access: the last one is moved back to end
//           with the row, and moved into place when it is used
//  kNarrow  shorter rows, element by element
// One kernel for each, because a branch between the loads makes the compiler wait for
// every one of them.
enum { kWhole = 0, kLoose = 1, kNarrow = 2 };

inline int row_mode(int n, int v) { return n % v == 0 ? kWhole : n >= v ? kLoose : kNarrow; }

// Calls f with a row_mode as a compile-time number.
template <typename F>
void with_mode(int mode, F f) {
  if (mode == kWhole) f(std::integral_constant<int, kWhole>{});
  else if (mode == kLoose) f(std::integral_constant<int, kLoose>{});
  else f(std::integral_constant<int, kNarrow>{});
}

// V elements of a row of n, from j on, as the words that memory holds; elements past
// the row are zeros. load() issues the accesses and get() uses them, so that a kernel
// can have several in flight. STREAM: nontemporal accesses, for rows that are touched
// once and whose accesses share no cache line (kWhole).
template <typename T, int V, int MODE, bool STREAM = false>
struct RowVec {
  static constexpr int kWords = V * (int)sizeof(T) / 4, kPer = kWords < 4 ? kWords : 4;
  typedef unsigned int Aligned __attribute__((ext_vector_type(kPer)));
  typedef Aligned Loose __attribute__((aligned(sizeof(T))));
  typedef typename std::conditional<MODE == kWhole, Aligned, Loose>::type Piece;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* __restrict__ row, int j, int n) {
    if (MODE == kNarrow) {
#pragma unroll
      for (int i = 0; i < V; ++i) set(i, row[min(j + i, n - 1)]);
      return;
    }
    const int at = MODE == kWhole ? (j < n ? j : 0) : min(j, n - V);
    const Piece* p = reinterpret_cast<const Piece*>(row + at);
#pragma unroll
    for (int i = 0; i < kWords / kPer; ++i) {
      const Aligned v = STREAM ? (Aligned)__builtin_nontemporal_load(p + i) : (Aligned)p[i];
#pragma unroll
      for (int k = 0; k < kPer; ++k) w[i * kPer + k] = v[k];
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // The words in place (zeros past the row).
  __device__ __forceinline__ void fix(int j, int n) {
    if (MODE == kWhole) {
      if (j >= n) zero();
      return;
    }
    if (MODE == kNarrow) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (j + i >= n) set(i, T(0));
      return;
    }
    const int sh = j - min(j, n - V);
    if (sh == 0) return;
    // towards the front by sh elements, a power of two at a time
    constexpr int kE = 4 / (int)sizeof(T);  // elements of a word
    if (sh >= V) {
      zero();
      return;
    }
    if (kE == 2 && (sh & 1)) {
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        w[i] = (w[i] >> 16) | (i + 1 < kWords ? w[i + 1 < kWords ? i + 1 : i] << 16 : 0u);
    }
    const int ws = sh / kE;
#pragma unroll
    for (int step = 1; step < kWords; step *= 2)
      if (ws & step) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = i + step < kWords ? w[i + step < kWords ? i + step : i] : 0u;
      }
  }
  __device__ __forceinline__ float at(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void get(float (&o)[V], int j, int n) {
    fix(j, n);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = at(i);
  }
  __device__ __forceinline__ void set(int i, float v) { w[i] = __float_as_uint(v); }
  __device__ __forceinline__ void set(int i, bf16_t v) {
    w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | ((uint32_t)v << 16) : v;
  }
  // Rounds to the row's type.
  __device__ __forceinline__ void put(const float (&o)[V]) {
    if (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(o[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void store(T* __restrict__ row, int j, int n) const {
    if (MODE == kWhole ? j < n : MODE == kLoose && j + V <= n) {
      Piece* p = reinterpret_cast<Piece*>(row + j);
#pragma unroll
      for (int i = 0; i < kWords / kPer; ++i) {
        Aligned v;
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = w[i * kPer + k];
        if (STREAM) __builtin_nontemporal_store((Piece)v, p + i);
        else p[i] = v;
      }
    } else if (MODE != kWhole) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (j + i < n) {
          if constexpr (sizeof(T) == 4) row[j + i] = __uint_as_float(w[i]);
          else row[j + i] = (bf16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
        }
    }
  }
};

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
