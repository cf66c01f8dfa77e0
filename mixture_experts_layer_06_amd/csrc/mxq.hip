// mxq.hip — MXFP4 quantisation (OCP microscaling, E2M1 elements): every 32
// consecutive values along the reduction share the scale 2^(s-127),
//   s = floor(log2 max|v|) - 2 + 127, clamped to [0, 254]  (2 = E2M1's largest
//       exponent); 127 for a block of zeros, 255 (NaN) for a block that holds
//       a NaN or an infinity (its codes are then 0);
//   code = the E2M1 value nearest to v * 2^(127-s), ties to the even code,
//       saturating at 6.
// The value a
// code and its scale stand for has two significant bits and is exact in
// bfloat16 (down to its subnormals); the quantisers write it on request.
//
// HBM-bound: each value is read once; codes, scales and (optionally) values
// are written once.
#include "tiles.h"

namespace moe {
namespace {

// The block's scale byte from the largest magnitude's binary32 bits.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  const int s = (int)(top >> 23) - 2;  // subnormal magnitudes clamp to 0 like the smallest normals
  return top == 0u ? 127u : top >= 0x7f800000u ? 255u : (uint32_t)(s < 0 ? 0 : s);
}
// 2^(s-127); s = 0 is subnormal, s = 255 NaN.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

// Eight values of a row as they were loaded: their largest magnitude's
// binary32 bits, and their codes under scale byte s, the first in the lowest
// nibble. The hardware conversion divides by 2^(s-127), taking s as the
// exponent field of its scale operand (so s = 0 is 2^-127), and rounds once.
template <typename T>
struct Eight;

template <>
struct Eight<bf16_t> {
  uint4 r;
  __device__ __forceinline__ void load(const bf16_t* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t d[4] = {r.x, r.y, r.z, r.w};
    u16x2_t m = {0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, d[k] & 0x7fff7fffu));
    return (uint32_t)(m.x > m.y ? m.x : m.y) << 16;
  }
  __device__ __forceinline__ uint32_t codes(uint32_t s) const {
    const float sc = __uint_as_float(s << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, r.x), sc, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, r.y), sc, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, r.z), sc, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, r.w), sc, 3);
    return s == 255u ? 0u : c;
  }
};

template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ uint32_t top() const {
    return max(max(max(mag_bits(a.x), mag_bits(a.y)), max(mag_bits(a.z), mag_bits(a.w))),
               max(max(mag_bits(b.x), mag_bits(b.y)), max(mag_bits(b.z), mag_bits(b.w))));
  }
  __device__ __forceinline__ uint32_t codes(uint32_t s) const {
    const float sc = __uint_as_float(s << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a.x, a.y, sc, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a.z, a.w, sc, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b.x, b.y, sc, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b.z, b.w, sc, 3);
    return s == 255u ? 0u : c;
  }
};

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
  Eight<T> v[2];
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
    if (t >= 0) v[p].load(x + t * H + h);
    else v[p].zero();
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int rl = (threadIdx.x >> 5) + p * 8, r = r0 + rl;
    uint32_t top = v[p].top();
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const uint32_t sb = mx_scale_byte(top);
    const uint32_t codes = v[p].codes(sb);
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
  float div[4], sc[4];  // the conversion's scale operand, and the scale
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) top = max(top, mag_bits(v[k][j]));
    sb[j] = mx_scale_byte(top);
    div[j] = __uint_as_float(sb[j] << 23);
    sc[j] = mx_scale(sb[j]);
  }
  uint32_t finite = 0;  // blocks with a NaN or an infinity have codes 0
#pragma unroll
  for (int j = 0; j < 4; ++j) finite |= sb[j] == 255u ? 0u : 0xffu << (8 * j);
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
    uint32_t codes = 0;  // byte j: column j's codes of rows 2k (low nibble) and 2k+1
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[2 * k][0], v[2 * k + 1][0], div[0], 0);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[2 * k][1], v[2 * k + 1][1], div[1], 1);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[2 * k][2], v[2 * k + 1][2], div[2], 2);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[2 * k][3], v[2 * k + 1][3], div[3], 3);
    codes &= finite;
    if (q != nullptr) *reinterpret_cast<uint32_t*>(q + (blk * 16 + k) * N + col) = codes;
    if (values != nullptr) {
      const f32x2_t p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 0),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 1),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 2),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 3)};
      float lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = p[j].x * sc[j];
        hi[j] = p[j].y * sc[j];
      }
      uint16_t* o = values + (blk * 32 + 2 * k) * N + col;
      *reinterpret_cast<uint2*>(o) = make_uint2(exact_bf16x2(lo[0], lo[1]), exact_bf16x2(lo[2], lo[3]));
      *reinterpret_cast<uint2*>(o + N) = make_uint2(exact_bf16x2(hi[0], hi[1]), exact_bf16x2(hi[2], hi[3]));
    }
  }
}

// ------------------------------------------------------------------ few-row product

// The grouped MXFP4 product where each expert has few rows (decode): bound by
// streaming the experts' packed weights once. A block takes one non-empty
// expert's 128 columns, its four waves a quarter of the reduction each (with
// few rows there are too few column groups to keep enough loads in flight),
// and the partial sums meet in LDS, added in wave order.
//
// A 16x16x128 MFMA operand holds, in lane 16q + i, the 32 reduction values of
// row i that are MX block q of the step, so a lane's fragment is exactly one
// block of its row: the lane loads those 32 values of x, takes their maximum
// and converts them without any exchange between lanes. For the weights a lane
// loads 16 packed rows (32 reduction values) of 8 columns and transposes the
// bytes in registers, fragment j being column 8i + j.
template <typename T>
__global__ __launch_bounds__(256, 2) void mx_stream_kernel(const T* __restrict__ x, RowMap gx,
                                                        const uint8_t* __restrict__ w,
                                                        const uint8_t* __restrict__ w_scale,
                                                        const int32_t* __restrict__ offsets, int e, int A, int Hin,
                                                        int N, int relu, bf16_t* __restrict__ out) {
  __shared__ int s_off[257];
  __shared__ int s_pre[257];
  __shared__ float s_acc[3][32][64];
  load_tile_prefix<0x40000000>(offsets, e, A, s_off, s_pre);  // s_pre[q]: non-empty experts before q
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ng = cdiv(N, 128);
  const int nth = blockIdx.x / ng;
  if (nth >= s_pre[e]) return;
  int lo = 0, hi = e - 1;  // largest expert with s_pre <= nth: the nth non-empty one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_pre[mid] <= nth) lo = mid;
    else hi = mid - 1;
  }
  const int ex = __builtin_amdgcn_readfirstlane(lo);
  const int r0 = s_off[ex], cnt = s_off[ex + 1] - r0;
  const int n0 = blockIdx.x % ng * 128;
  const int kq = lane >> 4, ci = lane & 15;
  const int col = n0 + 8 * ci;
  const int nsteps = Hin / 128;
  const int s0 = wave * nsteps / 4, s1 = (wave + 1) * nsteps / 4;
  const int n64 = (N + 63) & ~63;
  const uint32_t none = col < N ? 0u : kOOB;  // N is a multiple of 16
  const __amdgpu_buffer_rsrc_t wsrc = make_rsrc(w + (int64_t)ex * (Hin / 2) * N, (uint32_t)(Hin / 2) * (uint32_t)N);
  const __amdgpu_buffer_rsrc_t ssrc =
      make_rsrc(w_scale + (int64_t)ex * (Hin / 32) * n64, (uint32_t)(Hin / 32) * (uint32_t)n64);
  const uint32_t woff = (uint32_t)(16 * kq) * (uint32_t)N + (uint32_t)col;
  // scales of columns col + j (j = 0..7) are byte `sub` of 8 consecutive words
  const uint32_t soff = (uint32_t)kq * (uint32_t)n64 + (uint32_t)((col & ~63) + 32 * (ci & 1));
  const int sub = 8 * ((col & 63) >> 4);

  struct Set {
    uint2 w[16];
    uint4 sc[2];
  };
  for (int mc = 0; mc < cnt; mc += 16) {
    const int ml = mc + ci;
    int64_t t = -1;
    if (ml < cnt) t = gx.src != nullptr ? gather_src(gx, r0 + ml) : r0 + ml;
    const T* xp = x + (t >= 0 ? t : 0) * Hin + 32 * kq;
    auto load = [&](int step, Set& st) {
      // a step past this wave's share reads nothing new: zero weights, the last x again
      const uint32_t past = (step < s1 ? 0u : kOOB) | none;
      const uint32_t wk = woff + (uint32_t)(step < s1 ? step : s0) * 64u * (uint32_t)N;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        st.w[r] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(wsrc, (wk + (uint32_t)r * (uint32_t)N) | past, 0, 0));
      const uint32_t sk = soff + (uint32_t)(step < s1 ? step : s0) * 4u * (uint32_t)n64;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        st.sc[h] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(ssrc, (sk + 16u * h) | past, 0, 0));
    };
    // x of one step only: it is quantised before the next step's is loaded, and
    // each step's x is loaded ahead of its weights, so that quantising waits for
    // neither step's weights
    Eight<T> xr[4];
    auto load_x = [&](int step) {
      const int k = (step < s1 ? step : s1 - 1) * 128;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (t >= 0) xr[q].load(xp + k + 8 * q);
        else xr[q].zero();
      }
    };
    i32x8_t xf;
    int xs;
    auto quantise = [&]() {  // this lane's MX block: scale and codes
      const uint32_t sb = mx_scale_byte(max(max(xr[0].top(), xr[1].top()), max(xr[2].top(), xr[3].top())));
      xf = (i32x8_t){(int)xr[0].codes(sb), (int)xr[1].codes(sb), (int)xr[2].codes(sb), (int)xr[3].codes(sb),
                     0, 0, 0, 0};
      xs = (int)sb;
    };
    f32x4_t acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Set& st) {
      uint2 lo8[8], hi8[8];
      transpose_8x8_u8(st.w, lo8);
      transpose_8x8_u8(st.w + 8, hi8);
      const uint32_t ws[8] = {st.sc[0].x, st.sc[0].y, st.sc[0].z, st.sc[0].w,
                              st.sc[1].x, st.sc[1].y, st.sc[1].z, st.sc[1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const i32x8_t wf = {(int)lo8[j].x, (int)lo8[j].y, (int)hi8[j].x, (int)hi8[j].y, 0, 0, 0, 0};
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf, acc[j], 4, 4, 0, (int)(ws[j] >> sub), 0, xs);
      }
    };
    if (s0 < s1) {
      Set sa, sb;
      load_x(s0);
      load(s0, sa);
      for (int s = s0; s < s1; s += 2) {
        quantise();
        load_x(s + 1);
        load(s + 1, sb);
        __builtin_amdgcn_sched_barrier(0);
        multiply(sa);
        if (s + 1 >= s1) break;
        quantise();
        load_x(s + 2);
        load(s + 2, sa);
        __builtin_amdgcn_sched_barrier(0);
        multiply(sb);
      }
    }
    if (wave > 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) s_acc[wave - 1][j * 4 + r][lane] = acc[j][r];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float a = acc[j][r];
#pragma unroll
          for (int q = 0; q < 3; ++q) a += s_acc[q][j * 4 + r][lane];
          v[j] = relu && a < 0.f ? 0.f : a;
        }
        // fragment j's row 4 kq + r is column 8 (4 kq + r) + j
        const int n = n0 + 8 * (4 * kq + r);
        if (ml < cnt && n < N)
          *reinterpret_cast<uint4*>(out + (int64_t)(r0 + ml) * N + n) =
              make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
      }
    }
    __syncthreads();  // the sums have been read
  }
}

}  // namespace

moe_status launch_mx_stream(const void* x, moe_dtype dt, RowMap gx, const uint8_t* w, const uint8_t* w_scale,
                            const int32_t* offsets, int e, int A, int Hin, int N, moe_act act, void* out,
                            hipStream_t s) {
  const int relu = act == MOE_ACT_RELU;
  const int64_t grid = (int64_t)(e < A ? e : A) * cdiv(N, 128);
  if (dt == MOE_BF16)
    hipLaunchKernelGGL(mx_stream_kernel<bf16_t>, dim3((unsigned)grid), dim3(256), 0, s, (const bf16_t*)x, gx, w,
                       w_scale, offsets, e, A, Hin, N, relu, (bf16_t*)out);
  else
    hipLaunchKernelGGL(mx_stream_kernel<float>, dim3((unsigned)grid), dim3(256), 0, s, (const float*)x, gx, w,
                       w_scale, offsets, e, A, Hin, N, relu, (bf16_t*)out);
  return launch_status();
}

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
