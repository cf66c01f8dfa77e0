// norm.h — device helpers of the norms around a block, forward and backward.
#pragma once

#include "rows.h"

namespace moe {
namespace {

constexpr int kNV = 8;  // values per lane and access

// 8 values of a norm's weight or bias or a gate, in binary32 or bf16 (the same in all
// lanes), from j on; `none` where there is no such tensor.
template <int MODE>
__device__ __forceinline__ void load_w(const void* w, bool f32, int j, int n, float (&o)[kNV], float none) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < kNV; ++i) o[i] = none;
  } else if (f32) {
    RowVec<float, kNV, MODE> v;
    v.load((const float*)w, j, n);
    v.get(o, j, n);
  } else {
    RowVec<bf16_t, kNV, MODE> v;
    v.load((const bf16_t*)w, j, n);
    v.get(o, j, n);
  }
}
__device__ __forceinline__ float load_w1(const void* w, bool f32, int64_t j) {
  return f32 ? ((const float*)w)[j] : bf16_to_f32(((const bf16_t*)w)[j]);
}

// Q sums over the W waves of a row, the same in every lane. The two slots of s take
// turns (slot is toggled here), so that one barrier per call suffices: a slot is
// written again only behind the other slot's barrier, which every wave passes
// after its reads.
template <int W, int Q>
__device__ __forceinline__ void row_sums(float (&v)[Q], float (*s)[W][4], int wr, int& slot) {
#pragma unroll
  for (int q = 0; q < Q; ++q) v[q] = lanes_sum<kWave>(v[q]);
  if constexpr (W > 1) {
    if ((threadIdx.x & (kWave - 1)) == 0)
#pragma unroll
      for (int q = 0; q < Q; ++q) s[slot][wr][q] = v[q];
    __syncthreads();
    // every W lanes hold all waves' sums: one read and a few lane moves, no register
    // for each
    const f32x4_t all = *reinterpret_cast<const f32x4_t*>(s[slot][threadIdx.x % W]);
#pragma unroll
    for (int q = 0; q < Q; ++q) v[q] = lanes_sum<W>(all[q]);
    slot ^= 1;
  }
}

}  // namespace
}  // namespace moe
