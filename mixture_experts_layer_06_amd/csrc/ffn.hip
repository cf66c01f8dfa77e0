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
//  * ffn_pp_kernel (ffn_pp.hip; rows on 16 bytes, fp32 with enough tiles): tiles
//    of up to 256 x 256 filled by LDS DMA.
//  * ffn_tile_kernel (rows that are not 16-byte aligned, fp32 with few tiles):
//    tiles through registers into LDS, 16x16x32 bf16 or 16x16x4 fp32 MFMAs.
//  * glu_stream_kernel (bf16, a handful of rows over few tiles): the reduction
//    split over the waves of a block.
//  * glu_grad_kernel: the pointwise derivative, one pass over d, g and u.
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

// dg = d u act'(g), du = d act(g) in binary32, rounded once to the tensors' type
// and written side by side: row r of the output is dg's N columns, then du's, which
// the matrix products read as one (A, 2N) matrix. In bf16 that rounding adds to the
// result's own, so gradients are off by 2.4e-3 of their norm where one rounding
// gives 1.7e-3. It is taken because the bf16 MFMAs multiply bf16 operands: keeping
// dg and du whole means two bf16 terms of each and twice the products, the better
// part of the call's time; elementwise bf16 steps would round as often or more.
// fp32 tensors lose nothing here.
// HBM-bound: three reads and two writes, V elements (16 bytes) per lane and array,
// or one where N is no multiple of V (98304 x 1408 bf16: 239 to 265 us, 5.4 TB/s).
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
// multiplied, and writes them to LDS as memory has them. In a fragment lane
// 16q + i holds k values 8q .. 8q+7 of row i: one bf16 MFMA, or eight fp32 MFMAs
// whose step s takes k = 8q + s (any order of k serves, as long as both operands
// share it). From k-contiguous rows (16 bytes of padding) that is one or two
// 16-byte reads; from k rows two transposing bf16 reads (32-byte units swizzled
// over the banks) or, in fp32, one 4-byte read per step. 16-row fragments
// without rows are not multiplied.
template <typename T, int TM_, int TN_, int TK_, bool TOTALS>
struct TileCfg {
  typedef T Elem;
  static constexpr bool kTotals = TOTALS;
  static constexpr int kTM = TM_, kTN = TN_, kTK = TK_;
  static constexpr int kPitch = TK_ + 16 / (int)sizeof(T);  // elements; 16 bytes of padding
  static constexpr int kXB = TM_ * TK_ / 16 / 256, kWB = TN_ * TK_ / 16 / 256;  // 4 x 4 blocks per thread
  static constexpr int kFI = TM_ / 32, kFJ = TN_ / 32;                          // fragments per wave
  static_assert(kXB >= 1 && kWB >= 1 && kFI >= 1 && kFJ >= 2, "tile");
  // bytes of a k row of R columns
  static constexpr int row_pitch(int R) { return sizeof(T) == 2 ? R * 2 : (R + 4) * 4; }
  static constexpr int bytes(int R, bool k_rows) { return k_rows ? kTK * row_pitch(R) : R * kPitch * (int)sizeof(T); }
  // byte of column col of k row k
  static __device__ __forceinline__ int at(int R, int k, int col) {
    if (sizeof(T) == 4) return k * row_pitch(R) + col * 4;
    return k * row_pitch(R) + (((col >> 4) ^ unit_swz(R * 2, k)) * 32 + (col & 15) * 2);
  }
};

template <typename T>
struct __attribute__((aligned(4 * sizeof(T)))) Quad {
  T v[4];
};

// How a quad of a row of `n` elements is reached.
//  ALIGNED  every row starts on a multiple of four elements and has one.
//  LOOSE    any rows of at least four: an unaligned vector access (which the
//           hardware takes), moved back to stay inside the row at its end, the
//           value being shifted into place on its way to LDS.
//  SINGLE   element by element.
enum { ALIGNED = 0, LOOSE = 1, SINGLE = 2 };

template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) LooseQuad {
  T v[4];
};

template <typename T, int ACC>
__device__ __forceinline__ Quad<T> ld_quad(const unsigned char* base, uint32_t off) {
  if constexpr (ACC == ALIGNED) return *reinterpret_cast<const Quad<T>*>(base + off);
  return __builtin_bit_cast(Quad<T>, *reinterpret_cast<const LooseQuad<T>*>(base + off));
}
// Elements col .. col+3 of a row of n elements, 0 past its end.
template <typename T>
__device__ __forceinline__ Quad<T> ld_single(const T* row, int col, int n) {
  Quad<T> q = {};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (col + j < n) q.v[j] = row[col + j];
  return q;
}
// q without its first sh elements, zeros behind.
template <typename T>
__device__ __forceinline__ Quad<T> shifted(const Quad<T>& q, int sh) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_bit_cast(Quad<T>, sh >= 4 ? (uint64_t)0 : __builtin_bit_cast(uint64_t, q) >> (16 * sh));
  } else {
    Quad<T> r = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int k = j; k < 4; ++k) r.v[j] = sh == k - j ? q.v[k] : r.v[j];
    }
    return r;
  }
}

__device__ __forceinline__ int clamp_row(int v, int A) { return v < 0 ? 0 : (v > A ? A : v); }

template <class C, typename TO, int MODE, int ACC>
__global__ __launch_bounds__(256, 2) void ffn_tile_kernel(FfnCall c) {
  typedef typename C::Elem T;
  constexpr int kCols = MODE == GLU ? C::kTN / 2 : C::kTN;  // output columns per tile
  constexpr bool kFast = sizeof(T) == 2;
  __shared__ int s_off[257];
  __shared__ int s_pre[257];
  constexpr bool kXRows = MODE == WGRAD, kWRows = MODE != DGRAD;  // operand in k rows
  __shared__ __attribute__((aligned(16))) unsigned char s_x[C::bytes(C::kTM, kXRows)];
  __shared__ __attribute__((aligned(16))) unsigned char s_w[C::bytes(C::kTN, kWRows)];

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
    if (c.split > 1) {  // part blockIdx.y of the rows, in whole slices
      const int n = cdiv(K, C::kTK);
      const int a0 = (int)((int64_t)blockIdx.y * n / c.split), a1 = (int)((int64_t)(blockIdx.y + 1) * n / c.split);
      r0 += a0 * C::kTK;
      K = min(K - a0 * C::kTK, (a1 - a0) * C::kTK);
    }
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
  constexpr int kKC = C::kTK / 4, kES = sizeof(T);
  static_assert(256 % kKC == 0, "a thread's blocks share their k's (columns)");
  const int64_t wex = (int64_t)ex * c.Hin * c.ldw;
  const int nslice = cdiv(K, C::kTK);
  const int steps = nslice * (MODE == DGRAD ? c.npair : 1);
  const bool gat = MODE != DGRAD && c.rm.src != nullptr;
  const int ldx = MODE == DGRAD ? c.ldd : c.Hin, ldw = MODE == WGRAD ? c.ldd : c.ldw;

  // Byte offsets of this thread's quads from the slice's (scalar) bases: they
  // stay while whole slices are walked, so that a load costs no arithmetic. What
  // a row's or the reduction's end leaves to mend in a loaded quad (a shift, a
  // zero) is done on its way to LDS: touching it earlier would wait for it before
  // the slice at hand is multiplied. (3108 rows, 1001 -> 1501, 16 experts: GLU 336
  // us element by element, 102 mended at once, 55 so; 17535 rows, 1706 -> 1020, 8
  // experts: 498 mended at once, 215 so, 570 TFLOP/s.)
  const int kl = tid % kKC * 4;                                         // k of a k-contiguous operand's blocks
  const int wcol = tid % (C::kTN / 4) * 4, xcol = tid % (C::kTM / 4) * 4;  // column of the others'
  const int wn_ = n0 + (MODE == GLU ? wcol % kCols : wcol), xm_ = m0 + xcol;
  const int wc0 = kWRows ? max(min(wn_, NC - 4), 0) : 0, xc0 = kXRows ? max(min(xm_, M - 4), 0) : 0;
  // quads that straddle the end of a k row (columns behind it are not stored)
  const int wsh = kWRows && wn_ < NC ? wn_ - wc0 : 0, xsh = kXRows && xm_ < M ? xm_ - xc0 : 0;
  const bool wedge = __any(wsh > 0), xedge = __any(xsh > 0);
  uint32_t xo[C::kXB][4], wo[C::kWB][4];
  uint32_t xbad = 0;  // bit 4u + i: a gathered row of zeros
  int gi[C::kXB][4];  // WGRAD gather: row indexes of the slice to load next
  auto xk = [&](int u) { return (tid + u * 256) / (C::kTM / 4) * 4; };  // first local k of a block of k rows
  auto wk = [&](int u) { return (tid + u * 256) / (C::kTN / 4) * 4; };
#pragma unroll
  for (int u = 0; u < C::kXB; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (MODE == WGRAD) {
        xo[u][i] = (uint32_t)(xk(u) + i) * (uint32_t)(ldx * kES) + (uint32_t)(xc0 * kES);
      } else {
        const int ml = (tid + u * 256) / kKC * 4 + i;
        int row = ml < mrows ? ml : 0;
        if (gat) row = ml < mrows ? gather_src(c.rm, m0 + ml) : 0;
        if (row < 0) xbad |= 1u << (4 * u + i), row = 0;
        xo[u][i] = (uint32_t)row * (uint32_t)(ldx * kES) + (uint32_t)(kl * kES);
      }
    }
#pragma unroll
  for (int u = 0; u < C::kWB; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (MODE == DGRAD) {
        const int n = (tid + u * 256) / kKC * 4 + i;
        wo[u][i] = (uint32_t)(n0 + n < NC ? n : 0) * (uint32_t)(ldw * kES) + (uint32_t)(kl * kES);
      } else {
        wo[u][i] = (uint32_t)(wk(u) + i) * (uint32_t)(ldw * kES) + (uint32_t)(wc0 * kES);
      }
    }
  const bool xmend = __any(xbad != 0);
  // WGRAD gather: row v / div of x, or -1, the quotient by multiplication with
  // ceil(2^32 / div), which is exact or one too large for v < 2^31
  const uint32_t div = (uint32_t)c.rm.div, recip = 0xffffffffu / div + 1u;
  auto row_of = [&](int v) {
    uint32_t q = div == 1u ? (uint32_t)v : __umulhi((uint32_t)v, recip);
    if (q * div > (uint32_t)v) --q;
    return v >= 0 && q < (uint32_t)c.rm.rows ? (int)q : -1;
  };
  auto fetch_rows = [&](int step) {
#pragma unroll
    for (int u = 0; u < C::kXB; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = step * C::kTK + xk(u) + i;
        gi[u][i] = c.rm.src[r0 + (k < K ? k : 0)];
      }
  };
  if (MODE == WGRAD && gat && steps > 0) fetch_rows(0);

  Quad<T> xv[C::kXB][4], wv[C::kWB][4];
  auto load = [&](int step) {
    const int p = MODE == DGRAD ? step / nslice : pair;
    const int k0 = (MODE == DGRAD ? step % nslice : step) * C::kTK;
    const bool whole = k0 + C::kTK <= K;
    const T* x = reinterpret_cast<const T*>(MODE == DGRAD ? (p ? c.d[1] : c.d[0]) : c.x);
    const T* w = reinterpret_cast<const T*>(MODE == WGRAD ? (p ? c.d[1] : c.d[0]) : p ? c.w[1] : c.w[0]);
    if (MODE == GLU) w = reinterpret_cast<const T*>(wcol >= kCols ? c.w[1] : c.w[0]);
    w += MODE == WGRAD ? (int64_t)(r0 + k0) * ldw : MODE == GLU ? wex + (int64_t)k0 * ldw : wex + (int64_t)n0 * ldw;
    x += MODE == WGRAD ? (gat ? 0 : (int64_t)(r0 + k0) * ldx) : gat ? 0 : (int64_t)m0 * ldx;
    if constexpr (ACC == SINGLE) {
#pragma unroll
      for (int u = 0; u < C::kXB; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (MODE == WGRAD) {
            const int k = k0 + xk(u) + i;
            const int row = k >= K ? -1 : gat ? row_of(gi[u][i]) : xk(u) + i;
            xv[u][i] = row < 0 ? Quad<T>{} : ld_single<T>(x + (int64_t)row * ldx, xm_, M);
          } else {
            const T* row = x + (xo[u][i] - (uint32_t)(kl * kES)) / kES;
            xv[u][i] = xbad >> (4 * u + i) & 1 ? Quad<T>{} : ld_single<T>(row, k0 + kl, K);
          }
        }
#pragma unroll
      for (int u = 0; u < C::kWB; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (MODE == DGRAD)
            wv[u][i] = ld_single<T>(w + (wo[u][i] - (uint32_t)(kl * kES)) / kES, k0 + kl, K);
          else
            wv[u][i] = k0 + wk(u) + i < K ? ld_single<T>(w + (int64_t)(wk(u) + i) * ldw, wn_, NC) : Quad<T>{};
        }
    } else {
      // k-contiguous rows: from k0 on, or in the last slice moved back inside them
      const unsigned char* xb = reinterpret_cast<const unsigned char*>(x);
      const unsigned char* wb = reinterpret_cast<const unsigned char*>(w);
      const uint32_t back = (uint32_t)((min(k0 + kl, K - 4) - kl) * kES);
      if (MODE == WGRAD) {
        if (gat) {
          xbad = 0;
#pragma unroll
          for (int u = 0; u < C::kXB; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = row_of(gi[u][i]);
              if (row < 0) xbad |= 1u << (4 * u + i);
              xo[u][i] = (uint32_t)(row < 0 ? 0 : row) * (uint32_t)(ldx * kES) + (uint32_t)(xc0 * kES);
            }
        }
#pragma unroll
        for (int u = 0; u < C::kXB; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (whole || gat) xv[u][i] = ld_quad<T, ACC>(xb, xo[u][i]);
            else xv[u][i] = ld_quad<T, ACC>(xb, (uint32_t)min(xk(u) + i, K - 1 - k0) * (uint32_t)(ldx * kES) + (uint32_t)(xc0 * kES));
          }
      } else {
        if (whole) xb += (int64_t)k0 * kES;
#pragma unroll
        for (int u = 0; u < C::kXB; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) xv[u][i] = ld_quad<T, ACC>(xb, whole ? xo[u][i] : xo[u][i] + back);
      }
      if (MODE == DGRAD && whole) wb += (int64_t)k0 * kES;
#pragma unroll
      for (int u = 0; u < C::kWB; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (MODE == DGRAD) wv[u][i] = ld_quad<T, ACC>(wb, whole ? wo[u][i] : wo[u][i] + back);
          else if (whole) wv[u][i] = ld_quad<T, ACC>(wb, wo[u][i]);
          else wv[u][i] = ld_quad<T, ACC>(wb, (uint32_t)min(wk(u) + i, K - 1 - k0) * (uint32_t)(ldw * kES) + (uint32_t)(wc0 * kES));
        }
    }
    if (MODE == WGRAD && gat && step + 1 < steps) fetch_rows(step + 1);
  };
  // what the ends of rows and of the reduction leave to mend in the slice loaded
  auto mend = [&](int step) {
    if constexpr (ACC == SINGLE) return;
    const int k0 = (MODE == DGRAD ? step % nslice : step) * C::kTK;
    const bool whole = k0 + C::kTK <= K;
    const int ksh = k0 + kl - min(k0 + kl, K - 4);
    if (!whole || (MODE == WGRAD ? xedge || gat : xmend)) {
#pragma unroll
      for (int u = 0; u < C::kXB; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int sh = MODE == WGRAD ? (k0 + xk(u) + i < K ? xsh : 4) : ksh;
          if (xbad >> (4 * u + i) & 1) sh = 4;
          xv[u][i] = shifted<T>(xv[u][i], sh);
        }
    }
    if (!whole || (kWRows && wedge)) {
#pragma unroll
      for (int u = 0; u < C::kWB; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          wv[u][i] = shifted<T>(wv[u][i], MODE == DGRAD ? ksh : k0 + wk(u) + i < K ? wsh : 4);
    }
  };
  // block b of an operand with R rows (columns of k rows) to its LDS tile
  auto put = [&](unsigned char* t, const Quad<T>* v, int b, int R, bool k_rows) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int o = k_rows ? C::at(R, b / (R / 4) * 4 + i, b % (R / 4) * 4)
                           : ((b / kKC * 4 + i) * C::kPitch + b % kKC * 4) * (int)sizeof(T);
      *reinterpret_cast<Quad<T>*>(t + o) = v[i];
    }
  };
  // bf16 fragment of rows row .. row+15, k values kk + 8 kq ..
  auto frag = [&](const unsigned char* t, int R, int row, int kk, bool k_rows) {
    typedef short i16x4_t __attribute__((ext_vector_type(4)));
    typedef short i16x8_t __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;
    if (!k_rows) return *reinterpret_cast<const bf16x8_t*>(t + ((row + ci) * C::kPitch + kk + kq * 8) * 2);
    const unsigned char* p = t + C::at(R, kk + 8 * kq + (ci >> 2), row + (ci & 3) * 4);
    const i16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
    const i16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 4 * C::row_pitch(R)));
    return __builtin_bit_cast(bf16x8_t, (i16x8_t)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  // fp32 values k = kk + 8 kq + 4 h .. + 3 of row `row`
  auto four = [&](const unsigned char* t, int R, int row, int kk, int h, bool k_rows) {
    const int k = kk + 8 * kq + 4 * h;
    if (!k_rows) return *reinterpret_cast<const f32x4_t*>(t + (row * C::kPitch + k) * 4);
    f32x4_t v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const float*>(t + C::at(R, k + q, row));
    return v;
  };

  f32x4_t acc[C::kFI][C::kFJ];
#pragma unroll
  for (int i = 0; i < C::kFI; ++i)
#pragma unroll
    for (int j = 0; j < C::kFJ; ++j) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  // fp32 over long reductions: the sums of 128 k values at a time are added to
  // totals, which keeps the rounding from growing with the reduction (one running
  // sum over 4096 normal products is off by 1.1e-6 of the result's norm, this by
  // 2.3e-7)
  constexpr bool kTotals = C::kTotals;
  f32x4_t tot[kTotals ? C::kFI : 1][kTotals ? C::kFJ : 1];
  auto flush = [&](bool first) {
    if constexpr (kTotals) {
#pragma unroll
      for (int i = 0; i < C::kFI; ++i)
#pragma unroll
        for (int j = 0; j < C::kFJ; ++j) {
          tot[i][j] = first ? acc[i][j] : tot[i][j] + acc[i][j];
          acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        }
    }
  };
  flush(true);
  const int mw = wm * (C::kTM / 2);  // the wave's first row
  // LDS row of n fragment j: GLU's first half are gate columns, the others up columns
  auto wrow = [&](int j) {
    return MODE == GLU ? j / (C::kFJ / 2) * kCols + wn * (kCols / 2) + j % (C::kFJ / 2) * 16
                       : wn * (C::kTN / 2) + j * 16;
  };

  // lane: row m = ci of fragment i, columns 4 kq .. 4 kq + 3 of fragment j
  auto store = [&](TO* o, const float* v, int left) {  // left: columns that exist from o on
    if (left <= 0) return;
    Quad<TO> q;
#pragma unroll
    for (int r = 0; r < 4; ++r) from_f32(v[r], q.v[r]);
    if (ACC == ALIGNED) {
      *reinterpret_cast<Quad<TO>*>(o) = q;
    } else if (ACC == LOOSE && left >= 4) {
      *reinterpret_cast<LooseQuad<TO>*>(o) = __builtin_bit_cast(LooseQuad<TO>, q);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < left) o[r] = q.v[r];
    }
  };
  // Weight gradients: an expert may have any number of rows, and totals in
  // registers cost the large tiles a third of their occupancy, so there the sums
  // of an expert beyond kLongest rows leave in pieces of kPiece, each added to
  // the output by the lane that wrote the one before. So do the binary32 sums of
  // bf16 operands, whose MFMAs round once per 32 products. (fp32, one expert of 16421
  // rows among 64: off by 2.3e-6 of the norm as one sum, by 3.2e-7 so. 8192 rows,
  // 1001 x 1501, 8 experts of up to 1076 rows: 230 us as single sums, 318 with
  // totals in registers, 251 so; 16384 rows, 333 x 333, 64 experts, the longest of
  // 4802 rows: 476, 481, 560; where no expert is beyond 1024 rows nothing changes.)
  constexpr bool kPieces = MODE == WGRAD && sizeof(TO) == 4 && !kTotals;
  constexpr int kLongest = sizeof(T) == 4 ? 1024 : 4096, kPiece = sizeof(T) == 4 ? 256 : 4096;
  static_assert(kPiece % C::kTK == 0, "whole slices");
  bool held = false;  // the output holds the sums of earlier rows
  auto store_wgrad = [&]() __attribute__((always_inline)) {
    // opaque, so that no address is held in registers through the loop
    int ml = mw + ci, col = n0 + wrow(0) + 4 * kq;
    asm volatile("" : "+v"(ml), "+v"(col));
#pragma unroll
    for (int i = 0; i < C::kFI; ++i) {
      if (ml < mrows) {
        TO* const o = reinterpret_cast<TO*>(pair ? c.out[1] : c.out[0]) +
                      (((int64_t)blockIdx.y * c.e + ex) * c.Hin + m0 + ml) * c.ldw + col;
        // a row's earlier sums together, so that their loads overlap
        float v[C::kFJ][4];
#pragma unroll
        for (int j = 0; j < C::kFJ; ++j) {
          const int left = NC - (col + 16 * j);
#pragma unroll
          for (int r = 0; r < 4; ++r) v[j][r] = 0.f;
          if constexpr (kPieces) {
            if (held && left >= 4 && ACC != SINGLE) {
              const Quad<TO> q = ld_quad<TO, ACC>(reinterpret_cast<const unsigned char*>(o + 16 * j), 0);
#pragma unroll
              for (int r = 0; r < 4; ++r) v[j][r] = q.v[r];
            } else if (held) {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (r < left) v[j][r] = o[16 * j + r];
            }
          }
        }
#pragma unroll
        for (int j = 0; j < C::kFJ; ++j) {
#pragma unroll
          for (int r = 0; r < 4; ++r) v[j][r] = kPieces ? v[j][r] + acc[i][j][r] : acc[i][j][r];
          store(o + 16 * j, v[j], NC - (col + 16 * j));
        }
      }
      if (kPieces) {
#pragma unroll
        for (int j = 0; j < C::kFJ; ++j) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        asm volatile("" : "+v"(ml));
      }
      ml += 16;
    }
    held = true;
  };

  if (steps > 0) load(0);
  for (int s = 0; s < steps; ++s) {
    mend(s);
    __syncthreads();  // the slice before has been read
#pragma unroll
    for (int u = 0; u < C::kXB; ++u) put(s_x, xv[u], tid + u * 256, C::kTM, kXRows);
#pragma unroll
    for (int u = 0; u < C::kWB; ++u) put(s_w, wv[u], tid + u * 256, C::kTN, kWRows);
    __syncthreads();
    if (s + 1 < steps) load(s + 1);
#pragma unroll
    for (int kk = 0; kk < C::kTK; kk += 32) {
      if constexpr (sizeof(T) == 2) {
        bf16x8_t wb[C::kFJ];
#pragma unroll
        for (int j = 0; j < C::kFJ; ++j) wb[j] = frag(s_w, C::kTN, wrow(j), kk, kWRows);
#pragma unroll
        for (int i = 0; i < C::kFI; ++i) {
          if (mw + i * 16 >= mrows) continue;
          const bf16x8_t xa = frag(s_x, C::kTM, mw + i * 16, kk, kXRows);
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
            wb[j] = four(s_w, C::kTN, wrow(j) + ci, kk, h, kWRows);
#pragma unroll
          for (int i = 0; i < C::kFI; ++i) {
            if (mw + i * 16 >= mrows) continue;
            const f32x4_t xa = four(s_x, C::kTM, mw + i * 16 + ci, kk, h, kXRows);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int j = 0; j < C::kFJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(wb[j][q], xa[q], acc[i][j], 0, 0, 0);
          }
        }
      }
    }
    if (kTotals && (s + 1) * C::kTK % 128 == 0) flush(false);
    if (kPieces && c.pieces && K > kLongest && (s + 1) * C::kTK % kPiece == 0 && s + 1 < steps) store_wgrad();
  }

  if constexpr (kTotals) {
    flush(false);
#pragma unroll
    for (int i = 0; i < C::kFI; ++i)
#pragma unroll
      for (int j = 0; j < C::kFJ; ++j) acc[i][j] = tot[i][j];
  }

  if constexpr (MODE == WGRAD) {
    store_wgrad();
    return;
  }
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
        store(reinterpret_cast<TO*>(c.out[0]) + (int64_t)(m0 + ml) * NC + n, v, NC - n);
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
  const int64_t grid = tile_blocks<C, MODE>(c);
  if (grid > 0x7fffffff) return MOE_ERR_BAD_SHAPE;
  const dim3 blocks((unsigned)grid, MODE == WGRAD ? c.split : 1);
  if (c.Hin % 4 == 0 && c.N % 4 == 0 && c.ldw % 4 == 0)
    hipLaunchKernelGGL((ffn_tile_kernel<C, TO, MODE, ALIGNED>), blocks, dim3(256), 0, s, c);
  else if (c.Hin >= 4 && c.N >= 4)
    hipLaunchKernelGGL((ffn_tile_kernel<C, TO, MODE, LOOSE>), blocks, dim3(256), 0, s, c);
  else
    hipLaunchKernelGGL((ffn_tile_kernel<C, TO, MODE, SINGLE>), blocks, dim3(256), 0, s, c);
  return launch_status();
}

// 128 x 128 tiles where they give every CU one, else 32 x 64 with deep slices
// (more blocks, and more of the reduction in flight in each). The totals of
// long fp32 sums cost the large tiles a third of their occupancy (GLU of 4096
// rows, 1024 -> 1024, 8 experts: 264 us in place of 214), so those have them
// above 1024 k values only (running sums over 1024 are off by 6e-7). Weight
// gradients, whose sums are as long as an expert's rows, store pieces instead.
template <typename T, typename TO, int MODE>
moe_status launch_tile(const FfnCall& c, hipStream_t s) {
  constexpr bool kF32 = sizeof(T) == 4;
  typedef TileCfg<T, 128, 128, kF32 ? 32 : 64, false> Big;
  typedef TileCfg<T, 32, 64, 128, kF32> Small;
  if (tile_blocks<Big, MODE>(c) < device_cus()) return launch_cfg<Small, TO, MODE>(c, s);
  if constexpr (kF32 && MODE != WGRAD) {
    const int64_t k = MODE == GLU ? c.Hin : (int64_t)c.npair * c.N;
    if (k > 1024) return launch_cfg<TileCfg<T, 128, 128, 32, true>, TO, MODE>(c, s);
  }
  return launch_cfg<Big, TO, MODE>(c, s);
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
  if (glu_pp_takes(c) && c.dt == MOE_BF16 && glu_streams(c)) {
    const int64_t grid = (int64_t)(c.e < c.A ? c.e : c.A) * cdiv(c.N, 64);
    hipLaunchKernelGGL(glu_stream_kernel, dim3((unsigned)grid), dim3(512), 0, s, c);
    return launch_status();
  }
  if (glu_pp_takes(c)) return launch_glu_pp(c, s);
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
  if (dgrad_pp_takes(c)) return launch_dgrad_pp(c, s);
  return c.dt == MOE_F32 ? launch_tile<float, float, DGRAD>(c, s) : launch_tile<bf16_t, bf16_t, DGRAD>(c, s);
}


namespace {
// Parts the tile kernel splits every expert's rows into for weight gradients of
// few tiles and long experts: two blocks per CU, at least 512 rows each. (Before /
// after, us: 9001 rows, 265 x 137, one expert, fp32
// 173 / 31, bf16 90 / 21; 2171 rows, 103 x 64, fp32 39 / 18.)
int tile_split(const FfnCall& c) {
  typedef TileCfg<bf16_t, 128, 128, 64, false> Big;  // the sizes are those of fp32 as well
  typedef TileCfg<bf16_t, 32, 64, 128, false> Small;
  if (tile_blocks<Big, WGRAD>(c) >= device_cus()) return 1;
  const int64_t fill = 2 * device_cus() / tile_blocks<Small, WGRAD>(c), rows = c.A / c.e / 512;
  const int64_t S = fill < rows ? fill : rows;
  return S < 2 ? 1 : S > 16 ? 16 : (int)S;
}
// Sum of the partial weight gradients in part order: part (split, rows, npair * N)
// -> out[p] (rows, N of ld), one element per lane.
template <typename TO>
__global__ __launch_bounds__(256) void sum_tile_parts_kernel(const float* __restrict__ part, FfnCall c, int64_t total) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  float v = 0.f;
  for (int q = 0; q < c.split; ++q) v += part[q * total + i];
  const int cols = c.npair * c.N;
  const int64_t row = i / cols;
  const int col = (int)(i - row * cols);
  TO* o = reinterpret_cast<TO*>(col >= c.N ? c.out[1] : c.out[0]) + row * c.ldw + (col >= c.N ? col - c.N : col);
  from_f32(v, *o);
}
template <typename T>
moe_status launch_wgrad_parts(const FfnCall& c, moe_dtype out_dt, void* ws, hipStream_t s) {
  typedef TileCfg<T, 32, 64, 128, sizeof(T) == 4> Small;
  FfnCall p = c;
  p.ldw = c.npair * c.N;
  p.out[0] = ws;
  p.out[1] = (float*)ws + c.N;
  const moe_status st = launch_cfg<Small, float, WGRAD>(p, s);
  if (st != MOE_OK) return st;
  const int64_t total = (int64_t)c.e * c.Hin * p.ldw, grid = cdiv64(total, 256);
  if (grid > 0x7fffffff) return MOE_ERR_BAD_SHAPE;
  if (out_dt == MOE_F32)
    hipLaunchKernelGGL(sum_tile_parts_kernel<float>, dim3((unsigned)grid), dim3(256), 0, s, (const float*)ws, c, total);
  else
    hipLaunchKernelGGL(sum_tile_parts_kernel<bf16_t>, dim3((unsigned)grid), dim3(256), 0, s, (const float*)ws, c, total);
  return launch_status();
}
}  // namespace

// The larger of both kernels' needs: which one takes a call also hangs on its row strides.
size_t wgrad_ws_bytes(const FfnCall& c) {
  const int S = tile_split(c);
  const size_t tile = S > 1 ? (size_t)S * c.e * c.Hin * c.npair * c.N * sizeof(float) : 0;
  const size_t pp = wgrad_pp_takes(c) ? wgrad_pp_ws(c) : 0;
  return pp > tile ? pp : tile;
}

moe_status launch_wgrad(const FfnCall& c, moe_dtype out_dt, void* ws, hipStream_t s) {
  if (wgrad_pp_takes(c)) return launch_wgrad_pp(c, out_dt, ws, s);
  FfnCall p = c;
  p.split = tile_split(c);
  p.pieces = out_dt == MOE_F32;
  if (p.split > 1)
    return c.dt == MOE_F32 ? launch_wgrad_parts<float>(p, out_dt, ws, s) : launch_wgrad_parts<bf16_t>(p, out_dt, ws, s);
  if (c.dt == MOE_F32) return launch_tile<float, float, WGRAD>(p, s);
  return out_dt == MOE_F32 ? launch_tile<bf16_t, float, WGRAD>(p, s) : launch_tile<bf16_t, bf16_t, WGRAD>(p, s);
}

}  // namespace moe
