// mxq.hip — MXFP4 quantisation (OCP microscaling, E2M1 elements): every 32
// consecutive values along the reduction share the scale 2^(s-127),
//   s = floor(log2 max|v|) - 2 + 127, clamped to [0, 254]  (2 = E2M1's largest
//       exponent); 127 for a block of zeros, 255 (NaN) for a block that holds
//       a NaN or an infinity (its codes are then 0);
//   code = the E2M1 value nearest to v * 2^(127-s), ties to the even code,
//       saturating at 6.
// v * 2^(127-s) is exact in binary32 down to 2^-126, far below the smallest
// midpoint 0.25, so the hardware conversion of it rounds v once. The value a
// code and its scale stand for has two significant bits and is exact in
// bfloat16 (down to its subnormals); the quantisers write it on request.
//
// HBM-bound: each value is read once; codes, scales and (optionally) values
// are written once.
#include "common.h"

namespace moe {
namespace {

// The block's scale byte from the largest magnitude's binary32 bits.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  const int s = (int)(top >> 23) - 2;  // subnormal magnitudes clamp to 0 like the smallest normals
  return top == 0u ? 127u : top >= 0x7f800000u ? 255u : (uint32_t)(s < 0 ? 0 : s);
}
// 2^(127-s) for s <= 252, and 0 for the NaN scale: its codes are zeros.
__device__ __forceinline__ float mx_inv_scale(uint32_t s) {
  return s == 255u ? 0.f : __uint_as_float((254u - s) << 23);
}
// 2^(s-127); s = 0 is subnormal, s = 255 NaN.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

// v * inv with non-finite v (whose scale is NaN) as 0.
__device__ __forceinline__ float mx_scaled(float v, float inv) { return inv == 0.f ? 0.f : v * inv; }

// Codes of 8 scaled values, the first in the lowest nibble.
__device__ __forceinline__ uint32_t mx_codes8(const float v[8]) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], 1.f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], 1.f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], 1.f, 3);
  return r;
}

// bf16 pair of two exact values (their low 16 bits are zero).
__device__ __forceinline__ uint32_t exact_bf16x2(float lo, float hi) {
  return perm_b32(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));
// The values of codes 2K and 2K+1 of a word, times scale, as bf16.
template <int K>
__device__ __forceinline__ uint32_t mx_value_pair(uint32_t codes, float scale) {
  const f32x2_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, K);
  return exact_bf16x2(v.x * scale, v.y * scale);
}

// 8 consecutive elements at index i (a multiple of 8) as binary32.
template <typename T>
__device__ __forceinline__ void load8(const T* x, int64_t i, float v[8]) {
  if (sizeof(T) == 2) {
    const uint4 r = *reinterpret_cast<const uint4*>(x + i);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(x + i);
    const float4 b = *reinterpret_cast<const float4*>(x + i + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// ------------------------------------------------------------------ rows

// A block takes kRows rows of one 256-deep slice, 32 lanes (8 values each) per
// row, four lanes per scale block, so that its 16 x 8 scale bytes are one
// contiguous 128-byte piece of the slice-major scales.
constexpr int kRows = 16;

template <typename T>
__global__ __launch_bounds__(256) void mx_rows_kernel(const T* __restrict__ x, int x_rows, int H,
                                                      const int32_t* __restrict__ src, int div, int rows,
                                                      uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                      uint16_t* __restrict__ values) {
  __shared__ uint8_t s_sc[kRows * 8];
  const int slices = H / 256;
  const int slice = blockIdx.x % slices;
  const int r0 = blockIdx.x / slices * kRows;
  const int l = threadIdx.x & 31, h = slice * 256 + l * 8;
  float v[2][8];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int r = r0 + (threadIdx.x >> 5) + p * 8;
    int64_t t = -1;
    if (r < rows) {
      t = r;
      if (src != nullptr) {
        const int s = src[r];
        t = s >= 0 ? s / div : -1;
        if (t >= x_rows) t = -1;
      }
    }
    if (t >= 0) {
      load8(x, t * H + h, v[p]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[p][k] = 0.f;
    }
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int rl = (threadIdx.x >> 5) + p * 8, r = r0 + rl;
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, mag_bits(v[p][k]));
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const uint32_t sb = mx_scale_byte(top);
    const float inv = mx_inv_scale(sb);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[p][k] = mx_scaled(v[p][k], inv);
    const uint32_t codes = mx_codes8(v[p]);
    if ((l & 3) == 0) s_sc[rl * 8 + (l >> 2)] = (uint8_t)sb;
    if (r < rows) {
      const int64_t o = (int64_t)r * H + h;
      if (q != nullptr) *reinterpret_cast<uint32_t*>(q + o / 2) = codes;
      if (values != nullptr) {
        const float sc = mx_scale(sb);
        *reinterpret_cast<uint4*>(values + o) = make_uint4(mx_value_pair<0>(codes, sc), mx_value_pair<1>(codes, sc),
                                                           mx_value_pair<2>(codes, sc), mx_value_pair<3>(codes, sc));
      }
    }
  }
  if (scale == nullptr) return;
  __syncthreads();
  const int i = threadIdx.x;  // 4 bytes of the block's scales
  if (i < kRows * 2 && r0 + i / 2 < rows)
    *reinterpret_cast<uint32_t*>(scale + ((int64_t)slice * rows + r0) * 8 + i * 4) =
        *reinterpret_cast<const uint32_t*>(s_sc + i * 4);
}

// ------------------------------------------------------------------ weights

// A lane takes 4 columns of one block of 32 rows (16 lanes cover the 64
// columns of a scale group); codes leave as 4-byte pieces of the packed rows.
template <typename T>
__global__ __launch_bounds__(256) void mx_weights_kernel(const T* __restrict__ w, int Hin, int N,
                                                         uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                         uint16_t* __restrict__ values, int64_t tasks) {
  const int n64 = (N + 63) & ~63;
  const int groups = n64 / 64;
  const int lane = threadIdx.x & 63, c16 = lane & 15;
  // one task: a 64-column group of one block of rows; 4 per wave
  const int64_t task = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 4 + (lane >> 4);
  const bool live = task < tasks;
  const int64_t blk = live ? task / groups : 0;  // expert * (Hin/32) + block
  const int col = (int)(live ? task % groups : 0) * 64 + c16 * 4;
  const bool has = live && col < N;  // N is a multiple of 16
  float v[32][4];
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const T* p = w + (blk * 32 + k) * N + col;
    if (!has) {
      v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.f;
    } else if (sizeof(T) == 2) {
      const uint2 r = *reinterpret_cast<const uint2*>(p);
      v[k][0] = __uint_as_float(r.x << 16);
      v[k][1] = __uint_as_float(r.x & 0xffff0000u);
      v[k][2] = __uint_as_float(r.y << 16);
      v[k][3] = __uint_as_float(r.y & 0xffff0000u);
    } else {
      const float4 r = *reinterpret_cast<const float4*>(p);
      v[k][0] = r.x, v[k][1] = r.y, v[k][2] = r.z, v[k][3] = r.w;
    }
  }
  uint32_t sb[4];
  float inv[4], sc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) top = max(top, mag_bits(v[k][j]));
    sb[j] = mx_scale_byte(top);
    inv[j] = mx_inv_scale(sb[j]);
    sc[j] = mx_scale(sb[j]);
  }
  if (scale != nullptr) {
    // this lane's four bytes, and the interleaved word of columns c16 + 16 j
    const uint32_t own = has ? sb[0] | sb[1] << 8 | sb[2] << 16 | sb[3] << 24 : 0u;
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t from = (uint32_t)__shfl((int)own, (lane & 48) + 4 * j + (c16 >> 2));
      word |= (from >> (8 * (c16 & 3)) & 0xffu) << (8 * j);
    }
    if (live) *reinterpret_cast<uint32_t*>(scale + blk * n64 + (col & ~63) + 4 * c16) = word;
  }
  if (!has) return;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    uint32_t codes[2] = {0u, 0u};  // columns 0..3 of rows 2k (low nibbles) and 2k+1
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = mx_scaled(v[2 * k][j], inv[j]), b = mx_scaled(v[2 * k + 1][j], inv[j]);
      // byte j of the packed row: columns j's two codes
      codes[0] = j == 0   ? __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes[0], a, b, 1.f, 0)
                 : j == 1 ? __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes[0], a, b, 1.f, 1)
                 : j == 2 ? __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes[0], a, b, 1.f, 2)
                          : __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes[0], a, b, 1.f, 3);
    }
    if (q != nullptr) *reinterpret_cast<uint32_t*>(q + (blk * 16 + k) * N + col) = codes[0];
    if (values != nullptr) {
      float lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2_t p = j == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[0], 1.f, 0)
                          : j == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[0], 1.f, 1)
                          : j == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[0], 1.f, 2)
                                   : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[0], 1.f, 3);
        lo[j] = p.x * sc[j];
        hi[j] = p.y * sc[j];
      }
      uint16_t* o = values + (blk * 32 + 2 * k) * N + col;
      *reinterpret_cast<uint2*>(o) = make_uint2(exact_bf16x2(lo[0], lo[1]), exact_bf16x2(lo[2], lo[3]));
      *reinterpret_cast<uint2*>(o + N) = make_uint2(exact_bf16x2(hi[0], hi[1]), exact_bf16x2(hi[2], hi[3]));
    }
  }
}

}  // namespace

moe_status launch_mx_rows(const void* x, moe_dtype dt, int x_rows, int H, const int32_t* src, int div, int rows,
                          uint8_t* q, uint8_t* scale, uint16_t* values, hipStream_t s) {
  if (rows == 0) return MOE_OK;
  const int64_t grid = cdiv64(rows, kRows) * (H / 256);
  if (grid > 0x7fffffff) return MOE_ERR_BAD_SHAPE;
  if (dt == MOE_BF16)
    hipLaunchKernelGGL(mx_rows_kernel<bf16_t>, dim3((unsigned)grid), dim3(256), 0, s, (const bf16_t*)x, x_rows, H,
                       src, div, rows, q, scale, values);
  else
    hipLaunchKernelGGL(mx_rows_kernel<float>, dim3((unsigned)grid), dim3(256), 0, s, (const float*)x, x_rows, H,
                       src, div, rows, q, scale, values);
  return launch_status();
}

moe_status launch_mx_weights(const void* w, moe_dtype dt, int e, int Hin, int N, uint8_t* q, uint8_t* scale,
                             uint16_t* values, hipStream_t s) {
  const int64_t tasks = (int64_t)e * (Hin / 32) * cdiv(N, 64);
  const int64_t grid = cdiv64(tasks, 16);
  if (grid > 0x7fffffff) return MOE_ERR_BAD_SHAPE;
  if (dt == MOE_BF16)
    hipLaunchKernelGGL(mx_weights_kernel<bf16_t>, dim3((unsigned)grid), dim3(256), 0, s, (const bf16_t*)w, Hin, N, q,
                       scale, values, tasks);
  else
    hipLaunchKernelGGL(mx_weights_kernel<float>, dim3((unsigned)grid), dim3(256), 0, s, (const float*)w, Hin, N, q,
                       scale, values, tasks);
  return launch_status();
}

}  // namespace moe
