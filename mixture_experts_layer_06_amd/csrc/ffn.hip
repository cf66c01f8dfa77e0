// ffn.hip — the gated expert feed-forward and the grouped GEMM's gradients,
// over rows grouped by expert (rows offsets[ex] <= r < offsets[ex+1]):
//   GLU    out[r,n] = act(g) * u,  g = sum_h x[r,h] Wg[ex,h,n],
//                                  u = sum_h x[r,h] Wu[ex,h,n]
//   DGRAD  da[r,h]  = sum_p sum_n d_p[r,n] W_p[ex,h,n]
//   WGRAD  dW_p[ex,h,n] = sum_r x[r,h] d_p[r,n]   (r over the expert's rows)
// with p over one operand pair (a grouped GEMM) or two (the gated block's
// gate and up projections), and between them the gated block's pointwise
// derivative: with out's gradient d,  dg = d u act'(g),  du = d act(g).
//
// Each product is one matrix product per expert, "rows m" times "columns n"
// over a reduction k:
//            m              n             k       m operand      n operand
//   GLU      grouped row    N column      Hin     k contiguous   n contiguous
//   DGRAD    grouped row    Hin column    N       k contiguous   k contiguous
//   WGRAD    Hin row        N column      rows    m contiguous   n contiguous
// so the same tile kernel runs all three with different loads.
//
// Kernels
//  * ffn_pp_kernel (ffn_pp.hip; bf16 rows on 16 bytes): 256 x 256 tiles.
//  * ffn_tile_kernel (fp32, and bf16 shapes whose rows are not 16-byte
//    aligned): tiles through registers into LDS, 16x16x32 bf16 or 16x16x4
//    fp32 MFMAs.
//  * glu_stream_kernel (bf16, a handful of rows over few tiles): the reduction
//    split over the waves of a block.
//  * glu_grad_kernel: the pointwise derivative, one pass over d, g and u.
#include <atomic>

#include "tiles.h"

namespace moe {
namespace {

enum { GLU = 0, DGRAD = 1, WGRAD = 2 };

#include "act.h"


__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, bf16_t& o) { o = f32_to_bf16(v); }

// ------------------------------------------------------------------ pointwise derivative

// dg = d u act'(g), du = d act(g) in binary32, rounded once, written side by
// side: row r of the output is dg's N columns, then du's, which the matrix
// products read as one (A, 2N) matrix. HBM-bound: three reads and two writes,
// V elements (16 bytes) per lane and array, or one where N is no multiple of V.
template <typename T, int V, typename IDX>
__global__ __launch_bounds__(256) void glu_grad_kernel(const T* __restrict__ d, const T* __restrict__ g,
                                                       const T* __restrict__ u, IDX groups, int N, int act,
                                                       T* __restrict__ out) {
  constexpr bool kFast = sizeof(T) == 2;
  const IDX i = (IDX)blockIdx.x * 256 + threadIdx.x;
  if (i >= groups) return;
  const IDX per = (IDX)(N / V);  // groups of V elements per row
  const IDX row = i / per;
  const int64_t src = (int64_t)i * V;
  const int64_t dst = (int64_t)row * 2 * N + (int64_t)(i - row * per) * V;
  struct __attribute__((aligned(V * sizeof(T)))) Vec {
    T v[V];
  };
  const Vec dv = *reinterpret_cast<const Vec*>(d + src);
  const Vec gv = *reinterpret_cast<const Vec*>(g + src);
  const Vec uv = *reinterpret_cast<const Vec*>(u + src);
  Vec a, b;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    float av, slope;
    act_grad_of<kFast>(to_f32(gv.v[k]), act, av, slope);
    from_f32(to_f32(dv.v[k]) * to_f32(uv.v[k]) * slope, a.v[k]);
    from_f32(to_f32(dv.v[k]) * av, b.v[k]);
  }
  *reinterpret_cast<Vec*>(out + dst) = a;
  *reinterpret_cast<Vec*>(out + dst + N) = b;
}

template <typename T, int V>
moe_status launch_grad(const void* d, const void* g, const void* u, int64_t A, int N, int act, void* out,
                       hipStream_t s) {
  const int64_t groups = A * (N / V);
  const int64_t grid = cdiv64(groups, 256);
  if (grid > 0x7fffffff) return MOE_ERR_BAD_SHAPE;
  if (groups < (1ll << 31))  // 32-bit row division
    hipLaunchKernelGGL((glu_grad_kernel<T, V, uint32_t>), dim3((unsigned)grid), dim3(256), 0, s, (const T*)d,
                       (const T*)g, (const T*)u, (uint32_t)groups, N, act, (T*)out);
  else
    hipLaunchKernelGGL((glu_grad_kernel<T, V, uint64_t>), dim3((unsigned)grid), dim3(256), 0, s, (const T*)d,
                       (const T*)g, (const T*)u, (uint64_t)groups, N, act, (T*)out);
  return launch_status();
}

// ------------------------------------------------------------------ register-staged tiles

// Tiles of TM m rows x TN n rows (GLU: TN/2 columns of each projection), 4
// waves (2 x 2), TK-deep k slices. A thread carries 4 x 4 blocks of each
// operand per slice, prefetched into registers while the slice before is
// multiplied, and writes them to LDS k-contiguous (transposing them if memory
// has the other order). A lane reads k values 8q .. 8q+7 (q = lane / 16) of its
// row as one fragment: one bf16 MFMA, or eight fp32 MFMAs whose step s takes
// k = 8q + s (any order of k serves, as long as both operands share it).
// 16-row fragments without rows are not multiplied.
template <typename T, int TM_, int TN_, int TK_>
struct TileCfg {
  typedef T Elem;
  static constexpr int kTM = TM_, kTN = TN_, kTK = TK_;
  static constexpr int kPitch = TK_ + 16 / (int)sizeof(T);  // elements; 16 bytes of padding
  static constexpr int kXB = TM_ * TK_ / 16 / 256, kWB = TN_ * TK_ / 16 / 256;  // 4 x 4 blocks per thread
  static constexpr int kFI = TM_ / 32, kFJ = TN_ / 32;                          // fragments per wave
  static_assert(kXB >= 1 && kWB >= 1 && kFI >= 1 && kFJ >= 2, "tile");
};

template <typename T>
struct __attribute__((aligned(4 * sizeof(T)))) Quad {
  T v[4];
};

// Four elements at p, of which the first `avail` exist (the others are 0).
template <typename T, bool VEC>
__device__ __forceinline__ Quad<T> ld_quad(const T* p, int avail) {
  Quad<T> q = {};
  if (VEC) {
    if (avail > 0) q = *reinterpret_cast<const Quad<T>*>(p);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < avail) q.v[j] = p[j];
  }
  return q;
}

__device__ __forceinline__ int clamp_row(int v, int A) { return v < 0 ? 0 : (v > A ? A : v); }

// VEC: every row of every operand and output starts on a multiple of four
// elements and has a multiple of four.
template <class C, typename TO, int MODE, bool VEC>
__global__ __launch_bounds__(256) void ffn_tile_kernel(FfnCall c) {
  typedef typename C::Elem T;
  constexpr int kCols = MODE == GLU ? C::kTN / 2 : C::kTN;  // output columns per tile
  constexpr bool kFast = sizeof(T) == 2;
  __shared__ int s_off[257];
  __shared__ int s_pre[257];
  __shared__ __attribute__((aligned(16))) T s_x[C::kTM][C::kPitch];
  __shared__ __attribute__((aligned(16))) T s_w[C::kTN][C::kPitch];

  const int M = MODE == WGRAD ? c.Hin : 0;
  const int NC = MODE == DGRAD ? c.Hin : c.N;  // output columns
  int ex, m0, mrows, n0, pair = 0, r0 = 0, K;
  if (MODE == WGRAD) {
    const int ntn = cdiv(NC, kCols), ntm = cdiv(M, C::kTM);
    int b = blockIdx.x;
    n0 = b % ntn * kCols;
    b /= ntn;
    m0 = b % ntm * C::kTM;
    b /= ntm;
    pair = b % c.npair;
    ex = b / c.npair;
    mrows = min(C::kTM, M - m0);
    r0 = clamp_row(c.offsets[ex], c.A);
    K = clamp_row(c.offsets[ex + 1], c.A) - r0;
    if (K < 0) K = 0;
  } else {
    load_tile_prefix<C::kTM>(c.offsets, c.e, c.A, s_off, s_pre);
    Tile t;
    if (!pick_tile<C::kTM, kCols, 8>(s_off, s_pre, c.e, NC, blockIdx.x, t)) return;
    ex = t.ex;
    m0 = t.row0;
    mrows = t.rows;
    n0 = t.n0;
    K = MODE == GLU ? c.Hin : c.N;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int ci = lane & 15, kq = lane >> 4;
  // block b of a k-contiguous operand: k's 4 (b % kKC) .., rows 4 (b / kKC) ..;
  // of the others with R rows: rows 4 (b % (R/4)) .., k's 4 (b / (R/4)) ..
  constexpr int kKC = C::kTK / 4;
  const int64_t wex = (int64_t)ex * c.Hin * c.ldw;

  // rows of x this thread reads (GLU, DGRAD), -1: none
  int64_t xrow[C::kXB][4];
#pragma unroll
  for (int u = 0; u < C::kXB; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ml = (tid + u * 256) / kKC * 4 + i;
      xrow[u][i] = MODE == WGRAD || ml >= mrows ? -1 : MODE == GLU && c.rm.src ? gather_src(c.rm, m0 + ml) : m0 + ml;
    }
  const int nslice = cdiv(K, C::kTK);
  const int steps = nslice * (MODE == DGRAD ? c.npair : 1);

  Quad<T> xv[C::kXB][4], wv[C::kWB][4];
  auto load = [&](int step) {
    const int p = MODE == DGRAD ? step / nslice : pair;
    const int k0 = (MODE == DGRAD ? step % nslice : step) * C::kTK;
    const T* x = reinterpret_cast<const T*>(MODE == DGRAD ? (p ? c.d[1] : c.d[0]) : c.x);
#pragma unroll
    for (int u = 0; u < C::kXB; ++u) {
      const int b = tid + u * 256;
      if (MODE == WGRAD) {
        const int m = m0 + b % (C::kTM / 4) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // x rows k, columns m
          const int k = k0 + b / (C::kTM / 4) * 4 + i;
          const int64_t row = k >= K ? -1 : c.rm.src ? gather_src(c.rm, r0 + k) : r0 + k;
          xv[u][i] = ld_quad<T, VEC>(x + (row < 0 ? 0 : row) * c.Hin + m, row < 0 ? 0 : M - m);
        }
      } else {
        const int ldx = MODE == GLU ? c.Hin : c.ldd;
        const int k = k0 + b % kKC * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          xv[u][i] = ld_quad<T, VEC>(x + (xrow[u][i] < 0 ? 0 : xrow[u][i]) * ldx + k, xrow[u][i] < 0 ? 0 : K - k);
      }
    }
#pragma unroll
    for (int u = 0; u < C::kWB; ++u) {
      const int b = tid + u * 256;
      if (MODE == DGRAD) {
        const T* w = reinterpret_cast<const T*>(p ? c.w[1] : c.w[0]) + wex;
        const int k = k0 + b % kKC * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // weight rows n (= h), k contiguous
          const int n = n0 + b / kKC * 4 + i;
          wv[u][i] = ld_quad<T, VEC>(w + (int64_t)(n < NC ? n : 0) * c.ldw + k, n < NC ? K - k : 0);
        }
      } else {
        const int nl = b % (C::kTN / 4) * 4;
        const int half = MODE == GLU ? nl / kCols : pair;
        const int n = n0 + (MODE == GLU ? nl % kCols : nl);
        const T* w = MODE == GLU ? reinterpret_cast<const T*>(half ? c.w[1] : c.w[0]) + wex
                                 : reinterpret_cast<const T*>(half ? c.d[1] : c.d[0]) + (int64_t)r0 * c.ldd;
        const int64_t ld = MODE == GLU ? c.ldw : c.ldd;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = k0 + b / (C::kTN / 4) * 4 + i;
          wv[u][i] = ld_quad<T, VEC>(w + (k < K ? k : 0) * ld + n, k < K ? NC - n : 0);
        }
      }
    }
  };
  // block b of an operand with R rows to its LDS tile
  auto put = [&](T (*t)[C::kPitch], const Quad<T>* v, int b, int R, bool transposed) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!transposed) {
        *reinterpret_cast<Quad<T>*>(&t[b / kKC * 4 + i][b % kKC * 4]) = v[i];
      } else {
        Quad<T> q;
#pragma unroll
        for (int j = 0; j < 4; ++j) q.v[j] = v[j].v[i];
        *reinterpret_cast<Quad<T>*>(&t[b % (R / 4) * 4 + i][b / (R / 4) * 4]) = q;
      }
    }
  };

  f32x4_t acc[C::kFI][C::kFJ];
#pragma unroll
  for (int i = 0; i < C::kFI; ++i)
#pragma unroll
    for (int j = 0; j < C::kFJ; ++j) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  const int mw = wm * (C::kTM / 2);  // the wave's first row
  // LDS row of n fragment j: GLU's first half are gate columns, the others up columns
  auto wrow = [&](int j) {
    return MODE == GLU ? j / (C::kFJ / 2) * kCols + wn * (kCols / 2) + j % (C::kFJ / 2) * 16
                       : wn * (C::kTN / 2) + j * 16;
  };

  if (steps > 0) load(0);
  for (int s = 0; s < steps; ++s) {
    __syncthreads();  // the slice before has been read
#pragma unroll
    for (int u = 0; u < C::kXB; ++u) put(s_x, xv[u], tid + u * 256, C::kTM, MODE == WGRAD);
#pragma unroll
    for (int u = 0; u < C::kWB; ++u) put(s_w, wv[u], tid + u * 256, C::kTN, MODE != DGRAD);
    __syncthreads();
    if (s + 1 < steps) load(s + 1);
#pragma unroll
    for (int kk = 0; kk < C::kTK; kk += 32) {
      if constexpr (sizeof(T) == 2) {
        bf16x8_t wb[C::kFJ];
#pragma unroll
        for (int j = 0; j < C::kFJ; ++j) wb[j] = *reinterpret_cast<const bf16x8_t*>(&s_w[wrow(j) + ci][kk + kq * 8]);
#pragma unroll
        for (int i = 0; i < C::kFI; ++i) {
          if (mw + i * 16 >= mrows) continue;
          const bf16x8_t xa = *reinterpret_cast<const bf16x8_t*>(&s_x[mw + i * 16 + ci][kk + kq * 8]);
#pragma unroll
          for (int j = 0; j < C::kFJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], xa, acc[i][j], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4_t wb[C::kFJ];
#pragma unroll
          for (int j = 0; j < C::kFJ; ++j)
            wb[j] = *reinterpret_cast<const f32x4_t*>(&s_w[wrow(j) + ci][kk + kq * 8 + 4 * h]);
#pragma unroll
          for (int i = 0; i < C::kFI; ++i) {
            if (mw + i * 16 >= mrows) continue;
            const f32x4_t xa = *reinterpret_cast<const f32x4_t*>(&s_x[mw + i * 16 + ci][kk + kq * 8 + 4 * h]);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int j = 0; j < C::kFJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(wb[j][q], xa[q], acc[i][j], 0, 0, 0);
          }
        }
      }
    }
  }

  // lane: row m = ci of fragment i, columns 4 kq .. 4 kq + 3 of fragment j
  auto store = [&](TO* o, const float* v, int left) {  // left: columns that exist from o on
    if (VEC) {
      if (left <= 0) return;
      Quad<TO> q;
#pragma unroll
      for (int r = 0; r < 4; ++r) from_f32(v[r], q.v[r]);
      *reinterpret_cast<Quad<TO>*>(o) = q;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < left) from_f32(v[r], o[r]);
    }
  };
#pragma unroll
  for (int i = 0; i < C::kFI; ++i) {
    const int ml = mw + i * 16 + ci;
    if (ml >= mrows) continue;
#pragma unroll
    for (int j = 0; j < (MODE == GLU ? C::kFJ / 2 : C::kFJ); ++j) {
      const int n = n0 + wrow(j) + 4 * kq;
      if (MODE == GLU) {
        float v[4], g[4], u[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          g[r] = acc[i][j][r];
          u[r] = acc[i][j + C::kFJ / 2][r];
          v[r] = act_of<kFast>(g[r], c.act) * u[r];
        }
        const int64_t o = (int64_t)(m0 + ml) * NC + n;
        store(reinterpret_cast<TO*>(c.out[0]) + o, v, NC - n);
        if (c.out[1] != nullptr) {
          store(reinterpret_cast<TO*>(c.out[1]) + o, g, NC - n);
          store(reinterpret_cast<TO*>(c.out[2]) + o, u, NC - n);
        }
      } else {
        const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        TO* o = MODE == DGRAD ? reinterpret_cast<TO*>(c.out[0]) + (int64_t)(m0 + ml) * NC
                              : reinterpret_cast<TO*>(pair ? c.out[1] : c.out[0]) +
                                    ((int64_t)ex * c.Hin + m0 + ml) * c.ldw;
        store(o + n, v, NC - n);
      }
    }
  }
}

// Blocks of the tile kernel: an upper bound for GLU and DGRAD (surplus blocks exit).
template <class C, int MODE>
int64_t tile_blocks(const FfnCall& c) {
  const int nc = MODE == DGRAD ? c.Hin : c.N;
  constexpr int kCols = MODE == GLU ? C::kTN / 2 : C::kTN;
  if (MODE == WGRAD) return (int64_t)c.e * c.npair * cdiv(c.Hin, C::kTM) * cdiv(nc, kCols);
  return cdiv64((cdiv64(c.A, C::kTM) + (c.e < c.A ? c.e : c.A)) * cdiv(nc, kCols), 8) * 8;
}

template <class C, typename TO, int MODE>
moe_status launch_cfg(const FfnCall& c, hipStream_t s) {
  const bool vec = c.Hin % 4 == 0 && c.N % 4 == 0 && c.ldw % 4 == 0;
  const int64_t grid = tile_blocks<C, MODE>(c);
  if (grid > 0x7fffffff) return MOE_ERR_BAD_SHAPE;
  if (vec)
    hipLaunchKernelGGL((ffn_tile_kernel<C, TO, MODE, true>), dim3((unsigned)grid), dim3(256), 0, s, c);
  else
    hipLaunchKernelGGL((ffn_tile_kernel<C, TO, MODE, false>), dim3((unsigned)grid), dim3(256), 0, s, c);
  return launch_status();
}

// 128 x 128 tiles where they give every CU one, else 32 x 64 with deep slices
// (more blocks, and more of the reduction in flight in each).
template <typename T, typename TO, int MODE>
moe_status launch_tile(const FfnCall& c, hipStream_t s) {
  typedef TileCfg<T, 128, 128, sizeof(T) == 2 ? 64 : 32> Big;
  typedef TileCfg<T, 32, 64, 128> Small;
  if (tile_blocks<Big, MODE>(c) >= device_cus()) return launch_cfg<Big, TO, MODE>(c, s);
  return launch_cfg<Small, TO, MODE>(c, s);
}

// ------------------------------------------------------------------ few rows

// GLU for a handful of rows over few column tiles (the decode of one or a few
// sequences): bound by streaming the touched experts' weights, and even 64-column
// tiles would leave many CUs without one. A block takes 64 columns of one
// non-empty expert, its eight waves an eighth of the reduction each; the
// partial sums meet in LDS and are added in a fixed order. A lane loads 8 rows
// x 4 columns of each weight and transposes them in registers, so that MFMA
// j's row i is column 4i + j.
__global__ __launch_bounds__(512, 2) void glu_stream_kernel(FfnCall c) {
  __shared__ int s_off[257];
  __shared__ int s_pre[257];
  __shared__ f32x4_t s_acc[4][8][64];
  load_tile_prefix<0x40000000>(c.offsets, c.e, c.A, s_off, s_pre);  // s_pre[q]: non-empty experts before q
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ng = cdiv(c.N, 64);
  const int nth = blockIdx.x / ng;
  if (nth >= s_pre[c.e]) return;
  int lo = 0, hi = c.e - 1;  // largest expert with s_pre <= nth: the nth non-empty one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_pre[mid] <= nth) lo = mid;
    else hi = mid - 1;
  }
  const int ex = __builtin_amdgcn_readfirstlane(lo);
  const int r0 = s_off[ex], cnt = s_off[ex + 1] - r0;
  const int n0 = blockIdx.x % ng * 64;
  const int kq = lane >> 4, ci = lane & 15;
  const int ncol = n0 + 4 * ci;
  const int nsteps = cdiv(c.Hin, 32);
  const int s0 = wave * nsteps / 8, s1 = (wave + 1) * nsteps / 8;
  const uint32_t ldb = (uint32_t)c.ldw * 2u;
  const uint32_t bytes = ((uint32_t)(c.Hin - 1) * (uint32_t)c.ldw + (uint32_t)c.N) * 2u;
  const int64_t wex = (int64_t)ex * c.Hin * c.ldw;
  const __amdgpu_buffer_rsrc_t gsrc = make_rsrc(reinterpret_cast<const bf16_t*>(c.w[0]) + wex, bytes);
  const __amdgpu_buffer_rsrc_t usrc = make_rsrc(reinterpret_cast<const bf16_t*>(c.w[1]) + wex, bytes);
  const uint32_t none = ncol < c.N ? 0u : kOOB;
  const uint32_t woff = (uint32_t)(kq * 8) * ldb + (uint32_t)ncol * 2u;
  struct Set {
    uint2 g[8], u[8];
    uint4 x;
  };
  for (int mc = 0; mc < cnt; mc += 16) {
    int64_t t = -1;
    if (mc + ci < cnt) t = c.rm.src != nullptr ? gather_src(c.rm, r0 + mc + ci) : r0 + mc + ci;
    const bf16_t* xp = reinterpret_cast<const bf16_t*>(c.x) + (t < 0 ? 0 : t) * c.Hin;
    auto load = [&](int step, Set& st) {
      const uint32_t past = (step < s1 ? 0u : kOOB) | none;
      const uint32_t k = (uint32_t)(step < s1 ? step : s0) * 32u;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        st.g[r] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(gsrc, (woff + (k + r) * ldb) | past, 0, 0));
        st.u[r] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(usrc, (woff + (k + r) * ldb) | past, 0, 0));
      }
      const int kx = (int)k + kq * 8;  // Hin is a multiple of 8
      st.x = t >= 0 && step < s1 && kx < c.Hin ? *reinterpret_cast<const uint4*>(xp + kx) : make_uint4(0, 0, 0, 0);
    };
    f32x4_t ag[4], au[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) ag[j] = au[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Set& st) {
      const bf16x8_t xv = __builtin_bit_cast(bf16x8_t, st.x);
      uint4 cols[4];
      transpose_8x4_bf16(st.g, cols);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        ag[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, cols[j]), xv, ag[j], 0, 0, 0);
      transpose_8x4_bf16(st.u, cols);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        au[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, cols[j]), xv, au[j], 0, 0, 0);
    };
    if (s0 < s1) {
      Set sa, sb;
      load(s0, sa);
      for (int s = s0; s < s1; s += 2) {
        load(s + 1, sb);
        __builtin_amdgcn_sched_barrier(0);
        multiply(sa);
        if (s + 1 >= s1) break;
        load(s + 2, sa);
        __builtin_amdgcn_sched_barrier(0);
        multiply(sb);
      }
    }
    // waves 4-7 hand over to 0-3, which then each sum rows r = wave of all fragments
    if (wave >= 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s_acc[wave - 4][j][lane] = ag[j];
        s_acc[wave - 4][4 + j][lane] = au[j];
      }
    }
    __syncthreads();
    if (wave < 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s_acc[wave][j][lane] = ag[j] + s_acc[wave][j][lane];
        s_acc[wave][4 + j][lane] = au[j] + s_acc[wave][4 + j][lane];
      }
    }
    __syncthreads();
    if (wave < 4 && mc + ci < cnt) {
      float v[3][4];  // out, gate, up of columns n0 + 16 kq + 4 wave + j
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          g += reinterpret_cast<const float*>(&s_acc[q][j][lane])[wave];
          u += reinterpret_cast<const float*>(&s_acc[q][4 + j][lane])[wave];
        }
        v[0][j] = act_of<true>(g, c.act) * u;
        v[1][j] = g;
        v[2][j] = u;
      }
      const int n = n0 + 16 * kq + 4 * wave;  // N is a multiple of 8
      if (n < c.N) {
        const int64_t o = (int64_t)(r0 + mc + ci) * c.N + n;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (k == 0 || c.out[1] != nullptr)
            *reinterpret_cast<uint2*>(reinterpret_cast<bf16_t*>(c.out[k]) + o) =
                make_uint2(pack_bf16x2(v[k][0], v[k][1]), pack_bf16x2(v[k][2], v[k][3]));
      }
    }
    __syncthreads();  // the sums have been read
  }
}

}  // namespace

// Whether the call has few rows per expert and too few 64-column tiles for the
// CUs, so that the reduction is better split over a block's waves. Measured
// against the tile kernels: 132 tiles of depth 2048 16 us against 22, 192 of
// depth 4096 47 against 47, 224 of depth 4096 51 against 47.
static bool glu_streams(const FfnCall& c) {
  const int64_t experts = c.e < c.A ? c.e : c.A;
  return c.A <= 16 * experts && experts * cdiv(c.N, 64) * 4 < 3 * (int64_t)device_cus();
}

moe_status launch_glu(const FfnCall& c, hipStream_t s) {
  if (c.A == 0) return MOE_OK;
  if (ffn_pp_takes(c) && glu_streams(c)) {
    const int64_t grid = (int64_t)(c.e < c.A ? c.e : c.A) * cdiv(c.N, 64);
    hipLaunchKernelGGL(glu_stream_kernel, dim3((unsigned)grid), dim3(512), 0, s, c);
    return launch_status();
  }
  if (ffn_pp_takes(c)) return launch_glu_pp(c, s);
  return c.dt == MOE_F32 ? launch_tile<float, float, GLU>(c, s) : launch_tile<bf16_t, bf16_t, GLU>(c, s);
}

moe_status launch_glu_grad(const void* d, const void* g, const void* u, moe_dtype dt, int A, int N, moe_act act,
                           void* out, hipStream_t s) {
  if (A == 0) return MOE_OK;
  if (dt == MOE_F32)
    return N % 4 == 0 ? launch_grad<float, 4>(d, g, u, A, N, act, out, s)
                      : launch_grad<float, 1>(d, g, u, A, N, act, out, s);
  return N % 8 == 0 ? launch_grad<bf16_t, 8>(d, g, u, A, N, act, out, s)
                    : launch_grad<bf16_t, 1>(d, g, u, A, N, act, out, s);
}

moe_status launch_dgrad(const FfnCall& c, hipStream_t s) {
  if (c.A == 0) return MOE_OK;
  if (ffn_pp_takes(c)) return launch_dgrad_pp(c, s);
  return c.dt == MOE_F32 ? launch_tile<float, float, DGRAD>(c, s) : launch_tile<bf16_t, bf16_t, DGRAD>(c, s);
}

size_t wgrad_ws_bytes(const FfnCall& c) { return ffn_pp_takes(c) ? wgrad_pp_ws(c) : 0; }

moe_status launch_wgrad(const FfnCall& c, moe_dtype out_dt, void* ws, hipStream_t s) {
  if (ffn_pp_takes(c)) return launch_wgrad_pp(c, out_dt, ws, s);
  if (c.dt == MOE_F32) return launch_tile<float, float, WGRAD>(c, s);
  return out_dt == MOE_F32 ? launch_tile<bf16_t, float, WGRAD>(c, s) : launch_tile<bf16_t, bf16_t, WGRAD>(c, s);
}

}  // namespace moe
