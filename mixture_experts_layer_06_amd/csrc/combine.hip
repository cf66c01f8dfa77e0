// combine.hip — back to token order.
//  weighted: y[t] = sum_{k ascending} g[t,k] * y_perm[perm_dst[t*K+k]]
//            (y = sum_i g_i(x) E_i(x), SpMM page, section "MoE 模型与专家选择的挑战"),
//            fp32 sum, one rounding to the output type;
//  unweighted: out[t*K+k] = y_perm[perm_dst[t*K+k]]
//            (unpermuteOut = Unpermute(gmmY), "aclnnQuantGroupedMatMulAlltoAllv",
//            section 计算公式);
//  slot sum: y[t] = sum_{k ascending} z[t*K+k], the rows already in (t,k)
//            order and gated (by the GEMM's scattering epilogue).
// Both are pure bandwidth kernels: blocks over (output token, column
// stripe), 16-byte vector accesses when the row pitch allows, every input
// row read once (the weighted sum's loads and stores nontemporal). Few tokens (decode) get several column stripes per token,
// so that each thread issues the loads of all K rows of one vector at once.
#include "rows.h"

namespace moe {
namespace {

template <bool BF16, int VE>  // VE = elements per vector access
__global__ __launch_bounds__(256) void combine_weighted_kernel(const void* __restrict__ yp_,
                                                               const int32_t* __restrict__ perm_dst,
                                                               const float* __restrict__ gate, int T,
                                                               int K, int N, void* __restrict__ out_) {
  typedef typename std::conditional<BF16, bf16_t, float>::type E;
  const E* yp = reinterpret_cast<const E*>(yp_);
  E* out = reinterpret_cast<E*>(out_);
  const int nv = N / VE;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    int src[8];
    float g[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // no permutation: rows t*K+k in place; no gate: weight 1
      src[k] = k < K ? (perm_dst != nullptr ? perm_dst[(int64_t)t * K + k] : t * K + k) : 0;
      g[k] = k < K ? (gate != nullptr ? gate[(int64_t)t * K + k] : 1.f) : 0.f;
    }
    if (VE * sizeof(E) == 16) {
      // 16-byte vectors: the loads of all K rows are in flight before the
      // first is used; rows are read once and outputs written once, so both
      // are nontemporal
      typedef unsigned int u4 __attribute__((ext_vector_type(4)));
      for (int j = blockIdx.y * blockDim.x + threadIdx.x; j < nv; j += gridDim.y * blockDim.x) {
        u4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < K)
            v[k] = __builtin_nontemporal_load(reinterpret_cast<const u4*>(yp + (int64_t)src[k] * N + (int64_t)j * VE));
        float acc[VE];
#pragma unroll
        for (int q = 0; q < VE; ++q) acc[q] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k < K) {
            E e[VE];
            *reinterpret_cast<u4*>(e) = v[k];
#pragma unroll
            for (int q = 0; q < VE; ++q) {
              const float f = BF16 ? bf16_to_f32((bf16_t)e[q]) : (float)e[q];
              acc[q] = fmaf(g[k], f, acc[q]);
            }
          }
        }
        E o[VE];
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          if (BF16) o[q] = (E)f32_to_bf16(acc[q]);
          else o[q] = (E)acc[q];
        }
        __builtin_nontemporal_store(*reinterpret_cast<u4*>(o),
                                    reinterpret_cast<u4*>(out + (int64_t)t * N + (int64_t)j * VE));
      }
      continue;
    }
    for (int j = blockIdx.y * blockDim.x + threadIdx.x; j < nv; j += gridDim.y * blockDim.x) {
      float acc[VE];
#pragma unroll
      for (int q = 0; q < VE; ++q) acc[q] = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k < K) {
          const E* row = yp + (int64_t)src[k] * N + (int64_t)j * VE;
          E v[VE];
          if (VE * sizeof(E) == 16) {
            *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(row);
          } else {
#pragma unroll
            for (int q = 0; q < VE; ++q) v[q] = row[q];
          }
#pragma unroll
          for (int q = 0; q < VE; ++q) {
            const float f = BF16 ? bf16_to_f32((bf16_t)v[q]) : (float)v[q];
            acc[q] = fmaf(g[k], f, acc[q]);
          }
        }
      }
      E o[VE];
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        if (BF16) o[q] = (E)f32_to_bf16(acc[q]);
        else o[q] = (E)acc[q];
      }
      E* dst = out + (int64_t)t * N + (int64_t)j * VE;
      if (VE * sizeof(E) == 16) {
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<uint4*>(o);
      } else {
#pragma unroll
        for (int q = 0; q < VE; ++q) dst[q] = o[q];
      }
    }
  }
}

// Unpermute: one block per token copies its K rows. VB = bytes per access.
template <int VB>
__global__ __launch_bounds__(256) void unpermute_kernel(const unsigned char* __restrict__ yp,
                                                        const int32_t* __restrict__ perm_dst, int T,
                                                        int K, int64_t row_bytes,
                                                        unsigned char* __restrict__ out) {
  typedef typename std::conditional<VB == 16, uint4,
          typename std::conditional<VB == 8, uint2,
          typename std::conditional<VB == 4, uint32_t, uint16_t>::type>::type>::type V;
  const int64_t nv = row_bytes / VB;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k >= K) break;
      const int64_t i = (int64_t)t * K + k;
      const V* src = reinterpret_cast<const V*>(yp + (int64_t)perm_dst[i] * row_bytes);
      V* dst = reinterpret_cast<V*>(out + i * row_bytes);
      for (int64_t j = blockIdx.y * blockDim.x + threadIdx.x; j < nv; j += gridDim.y * blockDim.x)
        dst[j] = src[j];
    }
  }
}

// The weighted sum's gradient, with row p = perm_dst[t*K+k]:
//   dy_perm[p] = g[t,k] dout[t],  dgate[t,k] = sum_n dout[t,n] y_perm[p,n]
// HBM-bound, one pass: W waves take a token, hold a stretch of dout's row in
// registers and read and write all K rows' stretches of the same columns, every load
// of a stretch in flight before the first is used. A row that perm_dst puts outside
// [0, T*K) is neither read nor written, its gate's gradient 0. 16384 x 6 x 2048 bf16:
// 165 us, 5.3 TB/s, the rate of a copy.
template <typename E, int W, int MODE>
__global__ __launch_bounds__(256) void combine_bwd_kernel(const E* __restrict__ dout, const E* __restrict__ yp,
                                                          const int32_t* __restrict__ perm_dst,
                                                          const float* __restrict__ gate, int T, int K, int N,
                                                          E* __restrict__ dyp, float* __restrict__ dgate) {
  constexpr int V = 16 / sizeof(E);
  constexpr int kTok = 4 / W;
  typedef RowVec<E, V, MODE, MODE == kWhole> R;
  __shared__ float s[4][8];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int64_t t = (int64_t)blockIdx.x * kTok + wave / W;
  if (W == 1 && t >= T) return;  // W = 4: one token per block
  int64_t at[8];
  float g[8], dot[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int p = k < K ? perm_dst[t * K + k] : -1;
    at[k] = p >= 0 && p < (int64_t)T * K ? (int64_t)p * N : -1;
    g[k] = k < K ? gate[t * K + k] : 0.f;
    dot[k] = 0.f;
  }
  for (int j0 = wave % W * kWave * V; j0 < N; j0 += W * kWave * V) {
    const int j = j0 + lane * V;
    R d, y[8];
    d.load(dout + t * N, j, N);
    if (dgate != nullptr)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (at[k] >= 0) y[k].load(yp + at[k], j, N);
    float df[V];
    d.get(df, j, N);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (at[k] < 0) continue;
      if (dgate != nullptr) {
        float yf[V];
        y[k].get(yf, j, N);
#pragma unroll
        for (int i = 0; i < V; ++i) dot[k] = fmaf(df[i], yf[i], dot[k]);
      }
      if (dyp != nullptr) {
        float of[V];
#pragma unroll
        for (int i = 0; i < V; ++i) of[i] = g[k] * df[i];
        R o;
        o.put(of);
        o.store(dyp + at[k], j, N);
      }
    }
  }
  if (dgate == nullptr) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) dot[k] = lanes_sum<kWave>(dot[k]);
  if (W == 1) {
    float mine = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) mine = lane == k ? dot[k] : mine;
    if (lane < K) dgate[t * K + lane] = mine;
    return;
  }
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < 8; ++k) s[wave][k] = dot[k];
  __syncthreads();
  if (threadIdx.x < K) {
    float a = 0.f;
    for (int w = 0; w < 4; ++w) a += s[w][threadIdx.x];
    dgate[t * K + threadIdx.x] = a;
  }
}

}  // namespace

moe_status launch_combine_bwd(const void* dout, const void* y_perm, moe_dtype dt, const int32_t* perm_dst,
                              const float* gate, int T, int K, int N, void* dy_perm, float* dgate, hipStream_t s) {
  if (T == 0) return MOE_OK;
  // a wave per token where the tokens occupy the GPU or a wave spans the row (4096 x 2 x
  // 1024: 8.4 us, four waves 11.5; 1024 x 4 x 4096: 17.4 and 15; 512 x 4 x 2048: 7.4 and 5)
  const bool one = T >= 4096 || N <= (dt == MOE_BF16 ? 512 : 256);
  const dim3 grid((unsigned)(one ? cdiv(T, 4) : T));
  const auto go = [&](auto e, auto w, auto mode) {
    typedef decltype(e) E;
    hipLaunchKernelGGL((combine_bwd_kernel<E, w(), mode()>), grid, dim3(256), 0, s, (const E*)dout, (const E*)y_perm,
                       perm_dst, gate, T, K, N, (E*)dy_perm, dgate);
  };
  const auto by_width = [&](auto e, auto w) {
    with_mode(row_mode(N, 16 / sizeof(e)), [&](auto mode) {
      if constexpr (mode() != kNarrow || w() == 1) go(e, w, mode);
    });
  };
  const auto by_rows = [&](auto e) {
    if (one) by_width(e, std::integral_constant<int, 1>{});
    else by_width(e, std::integral_constant<int, 4>{});
  };
  if (dt == MOE_BF16) by_rows(bf16_t());
  else by_rows(float());
  return launch_status();
}

moe_status launch_combine(const void* y_perm, moe_dtype dt, const int32_t* perm_dst,
                          const float* gate, int T, int K, int N, void* out, hipStream_t s,
                          bool sum_slots) {
  if (T == 0) return MOE_OK;
  const bool bf = dt == MOE_BF16;
  if (sum_slots) {
    perm_dst = nullptr;
    gate = nullptr;
  }
  const bool weighted = gate != nullptr || sum_slots;
  // column stripes per token: one 256-vector stripe per block when tokens are few
  const int64_t vecs = weighted ? (bf ? N / 8 : N / 4) : (int64_t)N * (bf ? 2 : 4) / 16;
  int stripes = 1;
  if (T < 2048) {
    const int64_t st = (vecs + 255) / 256;
    stripes = st < 1 ? 1 : (st > 64 ? 64 : (int)st);
  }
  const dim3 grid(T < 65536 ? T : 65536, stripes);
  if (weighted) {
    if (bf) {
      if (N % 8 == 0)
        hipLaunchKernelGGL((combine_weighted_kernel<true, 8>), dim3(grid), dim3(256), 0, s, y_perm,
                           perm_dst, gate, T, K, N, out);
      else
        hipLaunchKernelGGL((combine_weighted_kernel<true, 1>), dim3(grid), dim3(256), 0, s, y_perm,
                           perm_dst, gate, T, K, N, out);
    } else {
      if (N % 4 == 0)
        hipLaunchKernelGGL((combine_weighted_kernel<false, 4>), dim3(grid), dim3(256), 0, s, y_perm,
                           perm_dst, gate, T, K, N, out);
      else
        hipLaunchKernelGGL((combine_weighted_kernel<false, 1>), dim3(grid), dim3(256), 0, s, y_perm,
                           perm_dst, gate, T, K, N, out);
    }
  } else {
    const int64_t rb = (int64_t)N * (bf ? 2 : 4);
    const unsigned char* src = (const unsigned char*)y_perm;
    unsigned char* dst = (unsigned char*)out;
    if (rb % 16 == 0)
      hipLaunchKernelGGL(unpermute_kernel<16>, dim3(grid), dim3(256), 0, s, src, perm_dst, T, K, rb, dst);
    else if (rb % 8 == 0)
      hipLaunchKernelGGL(unpermute_kernel<8>, dim3(grid), dim3(256), 0, s, src, perm_dst, T, K, rb, dst);
    else if (rb % 4 == 0)
      hipLaunchKernelGGL(unpermute_kernel<4>, dim3(grid), dim3(256), 0, s, src, perm_dst, T, K, rb, dst);
    else
      hipLaunchKernelGGL(unpermute_kernel<2>, dim3(grid), dim3(256), 0, s, src, perm_dst, T, K, rb, dst);
  }
  return launch_status();
}

}  // namespace moe
