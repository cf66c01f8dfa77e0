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

// The values of codes 2K (low half) and 2K+1 of a word under scale byte s, as
// bf16; NaN under 255.
template <int K>
__device__ __forceinline__ uint32_t mx_value_bits(uint32_t codes, uint32_t s) {
  const uint32_t v = __builtin_bit_cast(
      uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, __uint_as_float(s << 23), K));
  return s == 255u ? 0x7fc07fc0u : v;
}

// ------------------------------------------------------------------ rows

// A block takes kRows rows of one 256-deep slice, 32 lanes (8 values each) per
// row, four lanes per scale block, so that its 16 x 8 scale bytes are one
// contiguous 128-byte piece of the slice-major scales. (8192 x 7168 bf16 with
// values: 41 us, 6.5 TB/s; codes and scales alone 26 us, 5.7 TB/s.)
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
        *reinterpret_cast<uint4*>(values + o) = make_uint4(mx_value_bits<0>(codes, sb), mx_value_bits<1>(codes, sb),
                                                           mx_value_bits<2>(codes, sb), mx_value_bits<3>(codes, sb));
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

// Four columns of two consecutive rows as they were loaded.
template <typename T>
struct RowPair;

template <>
struct RowPair<bf16_t> {
  uint2 a, b;
  __device__ __forceinline__ void load(const unsigned char* p, uint32_t off, uint32_t pitch) {
    a = *reinterpret_cast<const uint2*>(p + off);
    b = *reinterpret_cast<const uint2*>(p + pitch + off);
  }
  // running maxima of the magnitudes' bits of columns 0..3
  struct Top {
    u16x2_t lo = {0, 0}, hi = {0, 0};
    __device__ __forceinline__ void add(const RowPair& r) {
      lo = __builtin_elementwise_max(lo, __builtin_bit_cast(u16x2_t, r.a.x & 0x7fff7fffu));
      hi = __builtin_elementwise_max(hi, __builtin_bit_cast(u16x2_t, r.a.y & 0x7fff7fffu));
      lo = __builtin_elementwise_max(lo, __builtin_bit_cast(u16x2_t, r.b.x & 0x7fff7fffu));
      hi = __builtin_elementwise_max(hi, __builtin_bit_cast(u16x2_t, r.b.y & 0x7fff7fffu));
    }
    __device__ __forceinline__ uint32_t bits(int j) const {
      return (uint32_t)(j == 0 ? lo.x : j == 1 ? lo.y : j == 2 ? hi.x : hi.y) << 16;
    }
  };
  __device__ __forceinline__ uint32_t codes(const float div[4]) const {  // byte j: column j, row a in the low nibble
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, perm_b32(b.x, a.x, 0x05040100u)), div[0], 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, perm_b32(b.x, a.x, 0x07060302u)), div[1], 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, perm_b32(b.y, a.y, 0x05040100u)), div[2], 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, perm_b32(b.y, a.y, 0x07060302u)), div[3], 3);
    return c;
  }
};

template <>
struct RowPair<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const unsigned char* p, uint32_t off, uint32_t pitch) {
    a = *reinterpret_cast<const float4*>(p + off);
    b = *reinterpret_cast<const float4*>(p + pitch + off);
  }
  struct Top {
    uint32_t t[4] = {0, 0, 0, 0};
    __device__ __forceinline__ void add(const RowPair& r) {
      t[0] = max(t[0], max(mag_bits(r.a.x), mag_bits(r.b.x)));
      t[1] = max(t[1], max(mag_bits(r.a.y), mag_bits(r.b.y)));
      t[2] = max(t[2], max(mag_bits(r.a.z), mag_bits(r.b.z)));
      t[3] = max(t[3], max(mag_bits(r.a.w), mag_bits(r.b.w)));
    }
    __device__ __forceinline__ uint32_t bits(int j) const { return t[j]; }
  };
  __device__ __forceinline__ uint32_t codes(const float div[4]) const {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a.x, b.x, div[0], 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a.y, b.y, div[1], 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a.z, b.z, div[2], 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a.w, b.w, div[3], 3);
    return c;
  }
};

// A lane takes 4 columns of one block of 32 rows (16 lanes cover the 64
// columns of a scale group, a wave four such tasks); codes leave as 4-byte
// pieces of the packed rows. Row k of every lane is at one scalar base plus
// the lane's own 32-bit offset, and values stay in their input type (per value
// 4 instructions in place of 15, which had made it instruction-bound). (8 x 7168
// x 2048 bf16: 53 us, 5.6 TB/s; with values 96 to 100 us, 5.3 to 5.5 TB/s.)
template <typename T>
__global__ __launch_bounds__(256) void mx_weights_kernel(const T* __restrict__ w, int Hin, int N,
                                                         uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                         uint16_t* __restrict__ values, int64_t tasks) {
  const int n64 = (N + 63) & ~63;
  const uint32_t groups = (uint32_t)n64 / 64;
  const int lane = threadIdx.x & 63, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t task0 = ((int64_t)blockIdx.x * 4 + wave) * 4;  // the wave's first task
  if (task0 >= tasks) return;
  const int64_t blk0 = task0 / groups;  // expert * (Hin/32) + block
  const uint32_t in = (uint32_t)(task0 - blk0 * groups) + (uint32_t)(lane >> 4);
  const uint32_t dblk = in / groups;  // blocks after the wave's first
  const bool live = task0 + (lane >> 4) < tasks;
  const int group = (int)(in - dblk * groups), col = group * 64 + c16 * 4;
  const bool has = live && col < N;  // N is a multiple of 16
  const uint32_t pitch = (uint32_t)N * (uint32_t)sizeof(T);
  // lanes without columns read the wave's first ones (in bounds, not used)
  const uint32_t off = has ? dblk * 32u * pitch + (uint32_t)col * (uint32_t)sizeof(T) : 0u;
  const unsigned char* base = reinterpret_cast<const unsigned char*>(w + blk0 * 32 * N);
  RowPair<T> v[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k].load(base + (int64_t)(2 * k) * pitch, off, pitch);
  typename RowPair<T>::Top top;
#pragma unroll
  for (int k = 0; k < 16; ++k) top.add(v[k]);
  uint32_t sb[4], finite = 0;  // blocks with a NaN or an infinity have codes 0
  float div[4];                // the conversions' scale operand
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sb[j] = mx_scale_byte(top.bits(j));
    div[j] = __uint_as_float(sb[j] << 23);
    finite |= sb[j] == 255u ? 0u : 0xffu << (8 * j);
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
    if (live) *reinterpret_cast<uint32_t*>(scale + (blk0 + dblk) * n64 + group * 64 + 4 * c16) = word;
  }
  if (!has) return;
  uint8_t* qb = q + blk0 * 16 * N;
  unsigned char* vb = reinterpret_cast<unsigned char*>(values + blk0 * 32 * N);
  const uint32_t qoff = dblk * 16u * (uint32_t)N + (uint32_t)col, voff = (dblk * 32u * (uint32_t)N + (uint32_t)col) * 2u;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const uint32_t codes = v[k].codes(div) & finite;
    if (q != nullptr) *reinterpret_cast<uint32_t*>(qb + (int64_t)k * N + qoff) = codes;
    if (values != nullptr) {
      const uint32_t p[4] = {mx_value_bits<0>(codes, sb[0]), mx_value_bits<1>(codes, sb[1]),
                             mx_value_bits<2>(codes, sb[2]), mx_value_bits<3>(codes, sb[3])};
      unsigned char* o = vb + (int64_t)(2 * k) * N * 2;
      *reinterpret_cast<uint2*>(o + voff) = make_uint2(perm_b32(p[1], p[0], 0x05040100u), perm_b32(p[3], p[2], 0x05040100u));
      *reinterpret_cast<uint2*>(o + 2 * (int64_t)N + voff) =
          make_uint2(perm_b32(p[1], p[0], 0x07060302u), perm_b32(p[3], p[2], 0x07060302u));
    }
  }
}

// ------------------------------------------------------------------ few-row product

// The grouped MXFP4 product where each expert has few rows (decode): bound by
// streaming the experts' packed weights once. A block takes one non-empty
// expert's 128 columns, its four waves a quarter of the reduction each (with
// few rows there are too few column groups to keep enough loads in flight),
// and the partial sums meet in LDS, added in wave order. (128 experts of 4096 x
// 1536, one row on average: 54 us, 5.1 TB/s of weights; two waves 55 to 65 us,
// eight 71. Three waves per SIMD spill, 79 us. A block of 32 rows and 64 columns
// in 4-byte loads takes 141 us at 12 rows per expert, where two passes of this
// take 113 and tiles 88.)
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
