// lora.hip — low-rank adapters of many requests beside a shared projection, over
// rows grouped by adapter (offsets[ex] <= r < offsets[ex+1], grouped row r being row
// t = rows[r] of the tensors, or r):
//   out[t] = base[t] + s_ex u[r] B_ex,  u[r] = x[t] A_ex
// and the gradients, with d = dout:
//   du[r] = s_ex d[t] B_ex^T,  dx[t] = base[t] + du[r] A_ex^T,
//   dA_ex = sum_r x[t]^T du[r],  dB_ex = s_ex sum_r u[r]^T d[t]
// A is (H,R), B (R,N), R at most 128: each product has one long side, so the calls
// are bound by the bytes of x, out, d and the adapters, not by the products.
//
//  * down_kernel: rows times a (K,R) matrix, K long. K is split over blocks (and
//    over a block's waves where tiles have 16 rows) until the GPU is occupied; the
//    binary32 partial sums go to the workspace. Matrices whose k rows are contiguous
//    pass through LDS, others are read as fragments directly.
//  * pack_kernel: adds the partial sums in order, applies the scale, and lays the
//    result out for its readers (rows, and transposed for the weight gradients).
//  * up_kernel: base plus u times an (R,N) matrix, which stays in registers while
//    rows pass by.
//  * grad_kernel: the weight gradients; a lane loads 8 rows of 16 bytes and
//    transposes them in registers, so that rows become the reduction.
//
// u and du are binary32. A bf16 MFMA takes them as two bf16 terms, u = hi + lo with
// lo = bf16(u - hi): 16 bits of u, so that a bf16 result carries one rounding, its
// own, where u rounded once to bf16 would add another of its size. The products
// double, which the memory's time hides. fp32 tensors use the fp32 MFMA.
//
// A fragment holds 8 consecutive k per lane (lane 16q + i: row or column i, k = 8q ..
// 8q+7): one bf16 16x16x32 MFMA, or eight fp32 16x16x4 ones, step s taking k = 8q + s.
#include "rows.h"
#include "tiles.h"

namespace moe {
namespace {

template <typename T>
struct Frag8;
template <>
struct Frag8<bf16_t> {
  typedef bf16x8_t Type;
};
template <>
struct Frag8<float> {
  struct Type {
    float v[8];
  };
};

__device__ __forceinline__ f32x4_t mma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma(const Frag8<float>::Type& a, const Frag8<float>::Type& b, f32x4_t c) {
#pragma unroll
  for (int s = 0; s < 8; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[s], b.v[s], c, 0, 0, 0);
  return c;
}

template <typename T, bool WHOLE, bool STREAM>
__device__ __forceinline__ typename Frag8<T>::Type frag_of(const RowVec<T, 8, WHOLE, STREAM>& v) {
  return __builtin_bit_cast(typename Frag8<T>::Type, v.w);
}

// u's 8 values as operands: the upper and lower bf16 terms, or the values.
__device__ __forceinline__ void split8(const float (&u)[8], bf16x8_t& hi, bf16x8_t& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = (__bf16)u[i];
    lo[i] = (__bf16)(u[i] - (float)hi[i]);
  }
}

__device__ __forceinline__ int row_at(const LoraCall& c, int r) {
  const int t = c.rows != nullptr ? c.rows[r] : r;
  return t >= 0 && t < c.T ? t : -1;
}

// ------------------------------------------------------------------ rows times (K,R)

// A tile: RW waves of XF fragments of 16 rows each, all F fragments of ranks; the
// other waves of the block (KW = 4 / RW teams) take other slices of k.
template <typename T, int F, int RW, int XF, bool WK>
struct DownCfg {
  static constexpr int kBM = RW * XF * 16, kKW = 4 / RW;
  // k of a slice: as deep as the loads in flight need and the ring's LDS allows
  static constexpr int kTK = RW == 1 ? (F * sizeof(T) >= 32 ? 32 : 64) : F * sizeof(T) >= 16 ? 64 : 128;
  static constexpr int kR = F * 16;                 // ranks, padded
  static constexpr int kPitch = sizeof(T) == 2 ? kR * 2 : (kR + 4) * 4;  // bytes of a k row in LDS
  static constexpr int kTile = kTK * kPitch;
  static constexpr int kTeam = 256 / kKW;           // threads
  static constexpr int kRing = WK ? 0 : kKW * 2 * kTile, kAcc = kKW > 1 ? 4 * F * kWave * 16 : 0;
  static constexpr int kLds = kRing > kAcc ? kRing : kAcc > 0 ? kAcc : 16;
};

template <typename T, int F, int RW, int XF, bool WK, bool WHOLE>
__global__ __launch_bounds__(256) void down_kernel(LoraCall c, const T* __restrict__ x, const T* __restrict__ w, int K,
                                                   int range, float* __restrict__ part) {
  typedef DownCfg<T, F, RW, XF, WK> C;
  typedef typename Frag8<T>::Type Frag;
  __shared__ int s_off[257], s_pre[257];
  __shared__ __attribute__((aligned(16))) unsigned char s_w[C::kLds];
  load_tile_prefix<C::kBM>(c.offsets, c.e, c.M, s_off, s_pre);
  if ((int)blockIdx.x >= s_pre[c.e]) return;
  Tile tile;
  tile_of<C::kBM, 1, 1>(s_off, s_pre, c.e, 1, blockIdx.x, tile);
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, ci = lane & 15, q = lane >> 4;
  const int team = wave / RW, rw = wave % RW, tt = threadIdx.x % C::kTeam;
  const int R = c.R;
  const T* we = w + (int64_t)tile.ex * K * R;
  const int k_lo = blockIdx.y * range, k_hi = min(K, k_lo + range);
  const int steps = cdiv(k_hi - k_lo, C::kTK * C::kKW);

  const T* xr[XF];  // rows that are not there read row 0 and become zeros
  bool there[XF];
#pragma unroll
  for (int i = 0; i < XF; ++i) {
    const int m = (rw * XF + i) * 16 + ci;
    const int t = m < tile.rows ? row_at(c, tile.row0 + m) : -1;
    there[i] = t >= 0;
    xr[i] = x + (int64_t)(there[i] ? t : 0) * K;
  }
  constexpr int kQ = C::kTK / 32;
  typedef RowVec<T, 8, WHOLE, WHOLE> X;
  X xv[XF][kQ];
  const auto load_x = [&](int k0) {
#pragma unroll
    for (int i = 0; i < XF; ++i)
#pragma unroll
      for (int s = 0; s < kQ; ++s) xv[i][s].load(xr[i], k0 + 32 * s + 8 * q, k_hi);
  };
  // a slice of the matrix in registers on its way to LDS: 8 ranks of a k row each
  constexpr int kPieces = C::kTK * C::kR / 8, kWV = kPieces > C::kTeam ? kPieces / C::kTeam : 1;
  static_assert(kPieces % C::kTeam == 0 || kPieces < C::kTeam, "whole pieces");
  typedef RowVec<T, 8, false> V;
  V wv[WK ? 1 : kWV];
  const auto piece_k = [&](int u) { return (tt + u * C::kTeam) / (C::kR / 8); };
  const auto piece_j = [&](int u) { return (tt + u * C::kTeam) % (C::kR / 8) * 8; };
  const auto load_w = [&](int k0) {
#pragma unroll
    for (int u = 0; u < kWV; ++u) wv[u].load(we + (int64_t)min(k0 + piece_k(u), k_hi - 1) * R, piece_j(u), R);
  };
  const auto put_w = [&](unsigned char* t, int k0) {
#pragma unroll
    for (int u = 0; u < kWV; ++u) {
      const int k = piece_k(u), j = piece_j(u);
      if (kPieces < C::kTeam && tt >= kPieces) continue;
      wv[u].fix(j, R);
      if (k0 + k >= k_hi) wv[u].zero();
      uint4* p = reinterpret_cast<uint4*>(t + k * C::kPitch + j * (int)sizeof(T));
      p[0] = make_uint4(wv[u].w[0], wv[u].w[1], wv[u].w[2], wv[u].w[3]);
      if constexpr (sizeof(T) == 4) p[1] = make_uint4(wv[u].w[4], wv[u].w[5], wv[u].w[6], wv[u].w[7]);
    }
  };
  f32x4_t acc[XF][F];
#pragma unroll
  for (int i = 0; i < XF; ++i)
#pragma unroll
    for (int f = 0; f < F; ++f) acc[i][f] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  unsigned char* ring = s_w + team * 2 * C::kTile;
  int k0 = k_lo + team * C::kTK;
  load_x(k0);
  if (!WK) {
    load_w(k0);
    put_w(ring, k0);
    __syncthreads();
  }
  for (int step = 0; step < steps; ++step, k0 += C::kTK * C::kKW) {
    Frag xf[XF][kQ];
#pragma unroll
    for (int i = 0; i < XF; ++i)
#pragma unroll
      for (int s = 0; s < kQ; ++s) {
        xv[i][s].fix(k0 + 32 * s + 8 * q, k_hi);
        if (!there[i]) xv[i][s].zero();
        xf[i][s] = frag_of(xv[i][s]);
      }
    RowVec<T, 8, WHOLE> wd[WK ? kQ : 1][WK ? F : 1];
    if constexpr (WK) {
#pragma unroll
      for (int s = 0; s < kQ; ++s)
#pragma unroll
        for (int f = 0; f < F; ++f)
          wd[s][f].load(we + (int64_t)min(16 * f + ci, R - 1) * K, k0 + 32 * s + 8 * q, k_hi);
    }
    const bool more = step + 1 < steps;
    if (more) {
      load_x(k0 + C::kTK * C::kKW);
      if constexpr (!WK) load_w(k0 + C::kTK * C::kKW);
    }
    const unsigned char* t = ring + (step & 1) * C::kTile;
#pragma unroll
    for (int s = 0; s < kQ; ++s)
#pragma unroll
      for (int f = 0; f < F; ++f) {
        Frag wf;
        if constexpr (WK) {
          wd[s][f].fix(k0 + 32 * s + 8 * q, k_hi);
          wf = frag_of(wd[s][f]);  // ranks past R repeat the last one; they are not stored
        } else if constexpr (sizeof(T) == 2) {
          typedef short i16x4_t __attribute__((ext_vector_type(4)));
          typedef short i16x8_t __attribute__((ext_vector_type(8)));
          typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;
          const unsigned char* p = t + (32 * s + 8 * q + (ci >> 2)) * C::kPitch + (16 * f + (ci & 3) * 4) * 2;
          const i16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
          const i16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 4 * C::kPitch));
          wf = __builtin_bit_cast(bf16x8_t, (i16x8_t)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            wf.v[i] = *reinterpret_cast<const float*>(t + (32 * s + 8 * q + i) * C::kPitch + (16 * f + ci) * 4);
        }
#pragma unroll
        for (int i = 0; i < XF; ++i) acc[i][f] = mma(wf, xf[i][s], acc[i][f]);
      }
    if (!WK && more) {
      put_w(ring + ((step + 1) & 1) * C::kTile, k0 + C::kTK * C::kKW);
      __syncthreads();
    }
  }
  // acc[i][f][r]: row ci of fragment i, rank 16f + 4q + r; teams are added in order
  if (C::kKW > 1) {
    f32x4_t* s_acc = reinterpret_cast<f32x4_t*>(s_w);
    __syncthreads();  // the ring is read no more
#pragma unroll
    for (int f = 0; f < F; ++f) s_acc[(wave * F + f) * kWave + lane] = acc[0][f];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int v = 1; v < 4; ++v) acc[0][f] += s_acc[(v * F + f) * kWave + lane];
  }
  float* dst = part + (int64_t)blockIdx.y * c.M * R;
#pragma unroll
  for (int i = 0; i < XF; ++i) {
    const int m = (rw * XF + i) * 16 + ci;
    if (m >= tile.rows) continue;
    float* row = dst + (int64_t)(tile.row0 + m) * R;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      RowVec<float, 4, false> o;
#pragma unroll
      for (int r = 0; r < 4; ++r) o.set(r, acc[i][f][r]);
      o.store(row, 16 * f + 4 * q, R);
    }
  }
}

// ------------------------------------------------------------------ partial sums

// u[r,j] = s sum_p part[p][r][j] (s the adapter's scale, or 1) to out (M,R), and
// transposed to tr, as grad_kernel reads it: (2,R16,pitch) bf16 terms or (R16,pitch)
// binary32, ranks past R zeros. Either may be null. Rows of no adapter are zeros in
// tr and stay as they were in out. A block takes 32 grouped rows, which lie side by
// side in every part; blockIdx.y selects one of two such jobs.
struct PackJob {
  const float* part;
  int parts;
  bool scaled;
  float* out;
  void* tr;
};
constexpr int kPackRows = 32;

template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(LoraCall c, PackJob j0, PackJob j1, int64_t pitch) {
  __shared__ float s_u[kPackRows * 129];
  __shared__ float s_scale[kPackRows];
  __shared__ int s_off[257];
  const PackJob job = blockIdx.y ? j1 : j0;
  const int r0 = blockIdx.x * kPackRows, R = c.R;
  const int rows = min(kPackRows, c.M - r0), n = rows * R;
  const int64_t slab = (int64_t)c.M * R;
  const float* src = job.part + (int64_t)r0 * R;
  // the parts' loads do not wait for the rows' adapters
  constexpr int kMost = kPackRows * 128 / 256;
  float a[kMost];
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int i = threadIdx.x + 256 * k;
    a[k] = 0.f;
    if (256 * k >= n) continue;
    if (i < n) {
#pragma unroll 8
      for (int p = 0; p < job.parts; ++p) a[k] += src[p * slab + i];
    }
  }
  for (int i = threadIdx.x; i <= c.e; i += 256) s_off[i] = min(max(c.offsets[i], 0), c.M);
  __syncthreads();
  const int covered = s_off[c.e] - r0;  // rows of some adapter
  if (threadIdx.x < kPackRows) {
    const int r = r0 + threadIdx.x;
    int lo = 0, hi = c.e - 1;  // the last adapter that starts at or before r
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_off[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    s_scale[threadIdx.x] = job.scaled && c.scale != nullptr ? c.scale[lo] : 1.f;
  }
  __syncthreads();
  const int live = min(n, max(covered, 0) * R);
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int i = threadIdx.x + 256 * k;
    if (i >= n) continue;
    const int r = i / R;
    const float v = i < live ? a[k] * s_scale[r] : 0.f;
    if (job.out != nullptr && i < live) job.out[(int64_t)r0 * R + i] = v;
    s_u[r * (R | 1) + i - r * R] = v;
  }
  if (job.tr == nullptr) return;
  __syncthreads();
  const int R16 = (R + 15) & ~15;
  for (int i = threadIdx.x; i < R16 * (kPackRows / 2); i += 256) {
    const int j = i / (kPackRows / 2), r = i % (kPackRows / 2) * 2;  // rows r, r + 1 of rank j; pitch holds whole blocks
    const float u0 = j < R && r < rows ? s_u[r * (R | 1) + j] : 0.f;
    const float u1 = j < R && r + 1 < rows ? s_u[(r + 1) * (R | 1) + j] : 0.f;
    const int64_t at = (int64_t)j * pitch + r0 + r;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float2*>((float*)job.tr + at) = make_float2(u0, u1);
    } else {
      const uint32_t hi = pack_bf16x2(u0, u1);
      const float l0 = u0 - __uint_as_float(hi << 16), l1 = u1 - __uint_as_float(hi & 0xffff0000u);
      *reinterpret_cast<uint32_t*>((bf16_t*)job.tr + at) = hi;
      *reinterpret_cast<uint32_t*>((bf16_t*)job.tr + R16 * pitch + at) = pack_bf16x2(l0, l1);
    }
  }
}

// ------------------------------------------------------------------ rows times (R,N)

constexpr int kUpRows = 64;   // rows of a tile
constexpr int kUpCols = 256;  // columns, 64 to a wave

// WS steps of 32 ranks; WS = 0: up to 16 ranks, the upper and lower terms of u side
// by side in one step (bf16). In a step lane (i, q) holds 8 ranks of columns 4i ..
// 4i+3 of the wave's 64, MFMA f taking column 4i + f as its row i: acc[f][r] of lane
// (row ci, q) is column 16q + 4r + f, 16 columns side by side.
template <typename T, int WS, bool WK, bool WHOLE>
__global__ __launch_bounds__(256) void up_kernel(LoraCall c, const float* __restrict__ u, int parts, bool scaled,
                                                 const T* __restrict__ w, int N, const T* base, T* out) {
  typedef typename Frag8<T>::Type Frag;
  typedef RowVec<T, 8, WHOLE, WHOLE> Y;
  constexpr int kS = WS > 0 ? WS : 1, kRF = kUpRows / 16;
  __shared__ int s_off[257], s_pre[257];
  load_tile_prefix<kUpRows>(c.offsets, c.e, c.M, s_off, s_pre);
  const int ntn = cdiv(N, kUpCols);
  const int total = s_pre[c.e] * ntn;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, ci = lane & 15, q = lane >> 4;
  const int R = c.R;
  Tile tile;
  bool idle = false;
  if ((int)blockIdx.x < total) {
    tile_of<kUpRows, kUpCols, 1>(s_off, s_pre, c.e, ntn, blockIdx.x, tile);
  } else {
    // rows of no adapter: base, or zeros
    if (base == out) return;
    const int L = blockIdx.x - total;
    tile.row0 = s_off[c.e] + L / ntn * kUpRows;
    tile.rows = min(kUpRows, c.M - tile.row0);
    tile.n0 = L % ntn * kUpCols;
    if (tile.rows <= 0) return;
    tile.ex = 0;
    idle = true;
  }
  const int n0 = tile.n0 + wave * 64;
  if (n0 >= N) return;
  const int n = n0 + 16 * q;
  // base's rows first: the longest way
  int t[kRF];
  Y b0[kRF], b1[kRF];
#pragma unroll
  for (int i = 0; i < kRF; ++i) t[i] = 16 * i + ci < tile.rows ? row_at(c, tile.row0 + 16 * i + ci) : -1;
  if (base != nullptr)
#pragma unroll
    for (int i = 0; i < kRF; ++i) {
      const T* row = base + (int64_t)max(t[i], 0) * N;
      b0[i].load(row, n, N);
      b1[i].load(row, n + 8, N);
    }
  Frag wf[kS][4];
  if (!idle) {
    const T* we = w + (int64_t)tile.ex * R * N;
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      const int j0 = WS > 0 ? 32 * s + 8 * q : 8 * (q & 1);
      if constexpr (WK) {
        RowVec<T, 8, false> v[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) v[f].load(we + (int64_t)min(n0 + 4 * ci + f, N - 1) * R, j0, R);
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          v[f].fix(j0, R);
          wf[s][f] = frag_of(v[f]);  // columns past N repeat the last one; they are not stored
        }
      } else {
        RowVec<T, 4, WHOLE> in[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) in[k].load(we + (int64_t)min(j0 + k, R - 1) * N, n0 + 4 * ci, N);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          in[k].fix(n0 + 4 * ci, N);
          if (j0 + k >= R) in[k].zero();
        }
        if constexpr (sizeof(T) == 2) {
          uint2 a[8];
          uint4 o[4];
#pragma unroll
          for (int k = 0; k < 8; ++k) a[k] = make_uint2(in[k].w[0], in[k].w[1]);
          transpose_8x4_bf16(a, o);
#pragma unroll
          for (int f = 0; f < 4; ++f) wf[s][f] = __builtin_bit_cast(bf16x8_t, o[f]);
        } else {
#pragma unroll
          for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int k = 0; k < 8; ++k) wf[s][f].v[k] = in[k].at(f);
        }
      }
    }
  }
  const float scale = scaled && c.scale != nullptr && !idle ? c.scale[tile.ex] : 1.f;
  const int64_t slab = (int64_t)c.M * R;
#pragma unroll
  for (int i = 0; i < kRF; ++i) {
    if (16 * i >= tile.rows) break;
    f32x4_t acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    if (!idle) {
      const float* ur = u + (int64_t)(tile.row0 + min(16 * i + ci, tile.rows - 1)) * R;
#pragma unroll
      for (int s = 0; s < kS; ++s) {
        const int j0 = WS > 0 ? 32 * s + 8 * q : 8 * (q & 1);
        float a[8];
        RowVec<float, 8, false> v;
        v.load(ur, j0, R);
        v.get(a, j0, R);
#pragma unroll 4
        for (int p = 1; p < parts; ++p) {
          float more[8];
          v.load(ur + p * slab, j0, R);
          v.get(more, j0, R);
#pragma unroll
          for (int k = 0; k < 8; ++k) a[k] += more[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] *= scale;
        if constexpr (sizeof(T) == 2) {
          bf16x8_t hi, lo;
          split8(a, hi, lo);
          if constexpr (WS > 0) {
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[f] = mma(wf[s][f], lo, acc[f]);
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[f] = mma(wf[s][f], hi, acc[f]);
          } else {
            const bf16x8_t both = q < 2 ? hi : lo;
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[f] = mma(wf[s][f], both, acc[f]);
          }
        } else {
          // up to 16 ranks: the upper lanes hold the same ranks again
          const bool on = WS > 0 || q < 2;
          Frag x;
#pragma unroll
          for (int k = 0; k < 8; ++k) x.v[k] = on ? a[k] : 0.f;
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[f] = mma(wf[s][f], x, acc[f]);
        }
      }
    }
    if (t[i] < 0) continue;
    float o0[8], o1[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      o0[k] = acc[k & 3][k >> 2];
      o1[k] = acc[k & 3][2 + (k >> 2)];
    }
    if (base != nullptr) {
      float v0[8], v1[8];
      b0[i].get(v0, n, N);
      b1[i].get(v1, n + 8, N);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        o0[k] += v0[k];
        o1[k] += v1[k];
      }
    }
    Y y0, y1;
    y0.put(o0);
    y1.put(o1);
    y0.store(out + (int64_t)t[i] * N, n, N);
    y1.store(out + (int64_t)t[i] * N, n + 8, N);
  }
}

// ------------------------------------------------------------------ weight gradients

// One of the two: for columns n of y (T,C) and ranks j,
//   g[n,j] = f_ex sum_r y[t_r][n] v[r][j]
// with v transposed in vt (pack_kernel's layout). Stored as (C,R) or, by_rank, (R,C).
struct GradSide {
  const void* y;
  const void* vt;
  int C;
  bool by_rank, scaled;
  void* out;
  float* part;  // split rows: (split, e, C, R) or (split, e, R, C) binary32
};

// A block takes CV x 16 columns (16 bytes a lane) of one adapter and one stretch of
// its rows, 32 rows to a wave and step; the waves' sums meet in LDS.
template <typename T, int F, bool WHOLE>
__global__ __launch_bounds__(256) void grad_kernel(LoraCall c, GradSide a, GradSide b, int tiles_a, int tiles_b,
                                                   int64_t pitch, int split, moe_dtype out_dt) {
  typedef typename Frag8<T>::Type Frag;
  constexpr int CV = 16 / (int)sizeof(T), kCols = CV * 16;
  __shared__ float s_acc[3 * F * kWave * 4 * CV];
  int L = blockIdx.x;
  const bool second = L >= tiles_a * c.e;
  if (second) L -= tiles_a * c.e;
  const int tiles = second ? tiles_b : tiles_a;
  const int C = second ? b.C : a.C;
  const T* y = (const T*)(second ? b.y : a.y);
  const T* vt = (const T*)(second ? b.vt : a.vt);
  const bool by_rank = second ? b.by_rank : a.by_rank;
  const int ex = L / tiles, n0 = L % tiles * kCols;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, ci = lane & 15, q = lane >> 4;
  const int R = c.R, R16 = (R + 15) & ~15, j0 = blockIdx.y * 16 * F;
  const int lo = min(max(c.offsets[ex], 0), c.M), hi = min(max(c.offsets[ex + 1], 0), c.M);
  const int len = max(hi - lo, 0), per = cdiv(cdiv(len, split), 128) * 128;
  const int r_lo = lo + blockIdx.z * per, r_hi = min(hi, r_lo + per);
  f32x4_t acc[CV][F];
#pragma unroll
  for (int v = 0; v < CV; ++v)
#pragma unroll
    for (int f = 0; f < F; ++f) acc[v][f] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  // Step by step: the row numbers two steps ahead, rows and v one step ahead of the
  // products.
  typedef RowVec<T, CV, WHOLE, WHOLE> X;
  constexpr int kTerms = sizeof(T) == 2 ? 2 : 1;
  X x[8];
  RowVec<T, 8, false> d[F][kTerms];
  RowVec<float, 8, false> at;
  int t[8];
  const int nc = n0 + CV * ci;
  const auto load_rows = [&](int r8) {
    if (c.rows != nullptr) at.load((const float*)c.rows, max(min(r8, r_hi - 1), 0), r_hi);
  };
  const auto use_rows = [&](int r8) {
    if (c.rows != nullptr) at.fix(max(min(r8, r_hi - 1), 0), r_hi);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int v = c.rows != nullptr ? (int)at.w[k] : r8 + k;
      t[k] = r8 + k < r_hi && v >= 0 && v < c.T ? v : -1;
    }
  };
  const auto load = [&](int r8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k].load(y + (int64_t)max(t[k], 0) * C, nc, C);
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int term = 0; term < kTerms; ++term) {
        const int j = min(j0 + 16 * f + ci, R16 - 1);
        d[f][term].load(vt + ((int64_t)term * R16 + j) * pitch, min(r8, r_hi - 1), r_hi);
      }
  };
  int r8 = r_lo + wave * 32 + 8 * q;  // this lane's 8 rows
  if (r_lo < r_hi) {
    load_rows(r8);
    use_rows(r8);
    load(r8);
    load_rows(r8 + 128);
  }
  for (int r0 = r_lo; r0 < r_hi; r0 += 128, r8 += 128) {
    Frag yf[CV], df[F][kTerms];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k].fix(nc, C);
      if (t[k] < 0) x[k].zero();
    }
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2 in[8];
        uint4 o[4];
#pragma unroll
        for (int k = 0; k < 8; ++k) in[k] = make_uint2(x[k].w[2 * h], x[k].w[2 * h + 1]);
        transpose_8x4_bf16(in, o);
#pragma unroll
        for (int v = 0; v < 4; ++v) yf[4 * h + v] = __builtin_bit_cast(bf16x8_t, o[v]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < CV; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) yf[v].v[k] = x[k].at(v);
    }
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int term = 0; term < kTerms; ++term) {
        d[f][term].fix(min(r8, r_hi - 1), r_hi);
        if (r8 >= r_hi) d[f][term].zero();
        df[f][term] = frag_of(d[f][term]);
      }
    if (r0 + 128 < r_hi) {
      use_rows(r8 + 128);
      load(r8 + 128);
      load_rows(r8 + 256);
    }
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int term = kTerms - 1; term >= 0; --term)
#pragma unroll
        for (int v = 0; v < CV; ++v) acc[v][f] = mma(yf[v], df[f][term], acc[v][f]);
  }
  // acc[v][f][r]: rank j0 + 16f + ci, column n0 + CV (4q + r) + v; the waves in order
  if (wave > 0)
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int v = 0; v < CV; ++v)
        *reinterpret_cast<f32x4_t*>(s_acc + ((((wave - 1) * F + f) * CV + v) * kWave + lane) * 4) = acc[v][f];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int v = 0; v < CV; ++v)
#pragma unroll
      for (int o = 0; o < 3; ++o)
        acc[v][f] += *reinterpret_cast<const f32x4_t*>(s_acc + (((o * F + f) * CV + v) * kWave + lane) * 4);
  float* part = second ? b.part : a.part;
  void* out = second ? b.out : a.out;
  const float fac = (second ? b.scaled : a.scaled) && c.scale != nullptr ? c.scale[ex] : 1.f;
  const int64_t base = ((int64_t)(part != nullptr ? blockIdx.z * c.e : 0) + ex) * C * R;
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int j = j0 + 16 * f + ci;
    if (j >= R) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int v = 0; v < CV; ++v) {
        const int n = n0 + CV * (4 * q + r) + v;
        if (n >= C) continue;
        const int64_t at = base + (by_rank ? (int64_t)j * C + n : (int64_t)n * R + j);
        const float g = fac * acc[v][f][r];
        if (part != nullptr) part[at] = g;
        else if (out_dt == MOE_F32) ((float*)out)[at] = g;
        else ((bf16_t*)out)[at] = f32_to_bf16(g);
      }
  }
}

// The sums of split rows, in order, of na values to oa and nb to ob.
__global__ __launch_bounds__(256) void grad_finish_kernel(const float* __restrict__ pa, int64_t na, void* oa,
                                                          const float* __restrict__ pb, int64_t nb, void* ob,
                                                          int split, moe_dtype out_dt) {
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool second = i >= na;
  if (second) i -= na;
  const int64_t n = second ? nb : na;
  if (i >= n) return;
  const float* part = second ? pb : pa;
  void* out = second ? ob : oa;
  float a = 0.f;
#pragma unroll 8
  for (int s = 0; s < split; ++s) a += part[s * n + i];
  if (out_dt == MOE_F32) ((float*)out)[i] = a;
  else ((bf16_t*)out)[i] = f32_to_bf16(a);
}

// ------------------------------------------------------------------ launches

int frags_of(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// Rows of a down tile: 128 where the adapters have at least 32 rows each on average,
// else 16; K is split until there are about two blocks per CU, in slices of at least
// 512.
struct DownPlan {
  bool small;
  int tiles, split, range;
};
DownPlan down_plan(int e, int M, int K) {
  DownPlan p;
  p.small = M < 32 * e || M < 64;
  const int bm = p.small ? 16 : 128;
  p.tiles = cdiv(M, bm) + (e < M ? e : M);          // at most
  const int likely = p.small ? (M < e ? M : cdiv(M, bm) + e / 2) : cdiv(M, bm) + e / 2;
  int split = 512 / (likely > 0 ? likely : 1);
  const int most = cdiv(K, 512);
  split = split < 1 ? 1 : split > most ? most : split;
  p.range = cdiv(cdiv(K, split), 256) * 256;
  p.split = cdiv(K, p.range);
  return p;
}

template <typename T, int F, bool WK>
void go_down(const LoraCall& c, const DownPlan& p, const void* x, const void* w, int K, float* part, hipStream_t s) {
  const dim3 grid(p.tiles, p.split);
  const auto go = [&](auto rw, auto whole) {
    hipLaunchKernelGGL((down_kernel<T, F, rw(), rw() == 1 ? 1 : 2, WK, whole()>), grid, dim3(256), 0, s, c,
                       (const T*)x, (const T*)w, K, p.range, part);
  };
  const auto by_width = [&](auto rw) {
    if (K % 8 == 0) go(rw, std::true_type{});
    else go(rw, std::false_type{});
  };
  if (p.small) by_width(std::integral_constant<int, 1>{});
  else by_width(std::integral_constant<int, 4>{});
}

template <typename T, bool WK>
void launch_down(const LoraCall& c, const DownPlan& p, const void* x, const void* w, int K, float* part,
                 hipStream_t s) {
  switch (frags_of(c.R)) {
    case 1: return go_down<T, 1, WK>(c, p, x, w, K, part, s);
    case 2: return go_down<T, 2, WK>(c, p, x, w, K, part, s);
    case 4: return go_down<T, 4, WK>(c, p, x, w, K, part, s);
    default: return go_down<T, 8, WK>(c, p, x, w, K, part, s);
  }
}

template <typename T, bool WK>
void launch_up(const LoraCall& c, const float* u, int parts, bool scaled, const void* w, int N, const void* base,
               void* out, hipStream_t s) {
  // the adapters' tiles, and as many again as rows of no adapter may need
  const dim3 grid((unsigned)((cdiv(c.M, kUpRows) + (c.e < c.M ? c.e : c.M) + 1) * cdiv(N, kUpCols)));
  const auto go = [&](auto ws, auto whole) {
    hipLaunchKernelGGL((up_kernel<T, ws(), WK, whole()>), grid, dim3(256), 0, s, c, u, parts, scaled, (const T*)w, N,
                       (const T*)base, (T*)out);
  };
  const auto by_width = [&](auto ws) {
    if (N % 8 == 0) go(ws, std::true_type{});
    else go(ws, std::false_type{});
  };
  if (c.R <= 16) by_width(std::integral_constant<int, 0>{});
  else if (c.R <= 32) by_width(std::integral_constant<int, 1>{});
  else if (c.R <= 64) by_width(std::integral_constant<int, 2>{});
  else by_width(std::integral_constant<int, 4>{});
}

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

struct FwdWs {
  size_t part, u, total;
};
// The up tiles of a row read its partial sums once per 256 columns: worth a launch
// that adds them where there are many of them.
bool pack_first(const DownPlan& p, int M, int R) { return p.split > 1 && (int64_t)M * R * p.split > 262144; }
FwdWs fwd_ws(int e, int M, int H, int R, bool keep) {
  const DownPlan p = down_plan(e, M, H);
  FwdWs w;
  w.part = 0;
  w.u = round256((size_t)p.split * M * R * 4);
  w.total = w.u + (!keep && pack_first(p, M, R) ? round256((size_t)M * R * 4) : 0);
  return w;
}

struct BwdWs {
  size_t part, du, dut, ut, ga, gb, total;
  int64_t pitch;
  int split;
};
// Rows of each adapter are split where the columns' blocks are fewer than two per
// CU, into stretches of at least 256 rows on average.
BwdWs bwd_ws(int es, int e, int M, int H, int N, int R) {
  const DownPlan p = down_plan(e, M, N);
  BwdWs w;
  const int R16 = (R + 15) & ~15, cols = 256 / es;
  w.pitch = (M + 63) / 64 * 64;
  w.part = 0;
  size_t o = round256((size_t)p.split * M * R * 4);
  w.du = o; o += round256((size_t)M * R * 4);
  const size_t tr = round256((size_t)R16 * w.pitch * 4);  // two bf16 terms, or binary32
  w.dut = o; o += tr;
  w.ut = o; o += tr;
  const int blocks = (cdiv(H, cols) + cdiv(N, cols)) * e * cdiv(R16, es == 2 ? 32 : 64);
  int split = 512 / blocks;
  const int most = M / e / 256;
  split = split > most ? most : split;
  w.split = split < 1 ? 1 : split;
  w.ga = o; o += w.split > 1 ? round256((size_t)w.split * e * H * R * 4) : 0;
  w.gb = o; o += w.split > 1 ? round256((size_t)w.split * e * R * N * 4) : 0;
  w.total = o;
  return w;
}

template <typename T>
moe_status run_fwd(const LoraCall& c, const void* x, const void* base, const void* a, const void* b, float* u_out,
                   void* out, unsigned char* ws, hipStream_t s) {
  const DownPlan p = down_plan(c.e, c.M, c.H);
  const FwdWs w = fwd_ws(c.e, c.M, c.H, c.R, u_out != nullptr);
  float* part = (float*)(ws + w.part);
  if (p.split == 1 && u_out != nullptr) part = u_out;
  launch_down<T, false>(c, p, x, a, c.H, part, s);
  int parts = p.split;
  if (p.split > 1 && (u_out != nullptr || pack_first(p, c.M, c.R))) {
    float* u = u_out != nullptr ? u_out : (float*)(ws + w.u);
    const PackJob job{part, parts, false, u, nullptr};
    hipLaunchKernelGGL(pack_kernel<T>, dim3(cdiv(c.M, kPackRows)), dim3(256), 0, s, c, job, job, (int64_t)0);
    part = u;
    parts = 1;
  }
  launch_up<T, false>(c, part, parts, true, b, c.N, base, out, s);
  return launch_status();
}

template <typename T>
moe_status run_bwd(const LoraCall& c, const void* dout, const void* x, const float* u, const void* a, const void* b,
                   const void* dx_base, void* dx, void* da, void* db, moe_dtype dw_dt, unsigned char* ws,
                   hipStream_t s) {
  const BwdWs w = bwd_ws(sizeof(T), c.e, c.M, c.H, c.N, c.R);
  float* part = (float*)(ws + w.part);
  float* du = (float*)(ws + w.du);
  if (c.M > 0) {
    // du, and transposed what the weight gradients multiply with
    const bool need = dx != nullptr || da != nullptr;
    const DownPlan p = down_plan(c.e, c.M, c.N);
    if (need) launch_down<T, true>(c, p, dout, b, c.N, part, s);
    const PackJob of_du{part, p.split, true, du, da != nullptr ? (void*)(ws + w.dut) : nullptr};
    const PackJob of_u{u, 1, false, nullptr, (void*)(ws + w.ut)};
    hipLaunchKernelGGL(pack_kernel<T>, dim3(cdiv(c.M, kPackRows), need && db != nullptr ? 2 : 1), dim3(256), 0, s, c,
                       need ? of_du : of_u, of_u, w.pitch);
  }
  if (c.M > 0 && dx != nullptr) launch_up<T, true>(c, du, 1, false, a, c.H, dx_base, dx, s);
  if (da == nullptr && db == nullptr) return launch_status();
  constexpr int cols = 256 / (int)sizeof(T);
  const int ta = da != nullptr ? cdiv(c.H, cols) : 0, tb = db != nullptr ? cdiv(c.N, cols) : 0;
  const GradSide ga{x, ws + w.dut, c.H, false, false, da, w.split > 1 ? (float*)(ws + w.ga) : nullptr};
  const GradSide gb{dout, ws + w.ut, c.N, true, true, db, w.split > 1 ? (float*)(ws + w.gb) : nullptr};
  // 32 ranks to a block (bf16: its 64 accumulators; with 128 the compiler spills some of
  // them, and drops the fourth value of a spilled sum), 64 in fp32
  constexpr int most = sizeof(T) == 2 ? 2 : 4;
  const int F = frags_of(c.R) > most ? most : frags_of(c.R);
  const dim3 grid((ta + tb) * c.e, cdiv((c.R + 15) / 16, F), w.split);
  const bool whole = c.H % (16 / sizeof(T)) == 0 && c.N % (16 / sizeof(T)) == 0;
  const auto go = [&](auto f) {
    if (whole)
      hipLaunchKernelGGL((grad_kernel<T, f(), true>), grid, dim3(256), 0, s, c, ga, gb, ta, tb, w.pitch, w.split,
                         dw_dt);
    else
      hipLaunchKernelGGL((grad_kernel<T, f(), false>), grid, dim3(256), 0, s, c, ga, gb, ta, tb, w.pitch, w.split,
                         dw_dt);
  };
  if (F == 1) go(std::integral_constant<int, 1>{});
  else if (F == 2 || most == 2) go(std::integral_constant<int, 2>{});
  else go(std::integral_constant<int, most>{});
  if (w.split > 1) {
    const int64_t na = da != nullptr ? (int64_t)c.e * c.H * c.R : 0, nb = db != nullptr ? (int64_t)c.e * c.R * c.N : 0;
    hipLaunchKernelGGL(grad_finish_kernel, dim3((unsigned)cdiv64(na + nb, 256)), dim3(256), 0, s, ga.part, na, da,
                       gb.part, nb, db, w.split, dw_dt);
  }
  return launch_status();
}

}  // namespace

size_t lora_ws_bytes(int e, int M, int H, int N, int R, bool keep) {
  return M > 0 ? fwd_ws(e, M, H, R, keep).total : 0;
}

size_t lora_bwd_ws_bytes(moe_dtype dt, int e, int M, int H, int N, int R) {
  return M > 0 ? bwd_ws(dtype_size(dt), e, M, H, N, R).total : 0;
}

moe_status launch_lora(const LoraCall& c, const void* x, const void* base, moe_dtype dt, const void* a, const void* b,
                       float* u_out, void* out, void* ws, hipStream_t s) {
  if (dt == MOE_F32) return run_fwd<float>(c, x, base, a, b, u_out, out, (unsigned char*)ws, s);
  return run_fwd<bf16_t>(c, x, base, a, b, u_out, out, (unsigned char*)ws, s);
}

moe_status launch_lora_bwd(const LoraCall& c, const void* dout, const void* x, const float* u, moe_dtype dt,
                           const void* a, const void* b, const void* dx_base, void* dx, void* da, void* db,
                           moe_dtype dw_dt, void* ws, hipStream_t s) {
  if (dt == MOE_F32)
    return run_bwd<float>(c, dout, x, u, a, b, dx_base, dx, da, db, dw_dt, (unsigned char*)ws, s);
  return run_bwd<bf16_t>(c, dout, x, u, a, b, dx_base, dx, da, db, dw_dt, (unsigned char*)ws, s);
}

}  // namespace moe
