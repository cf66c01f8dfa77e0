// loss.hip — the losses that train a router, and their gradient.
//
// With p_t = softmax(scores[t]), lse_t the logarithm of its sum, c_e how often
// expert e was chosen, n the live tokens and P_e the mean of p_te over them:
//   balance = E / (n K) sum_e c_e P_e        (1 where both are uniform)
//   z       = 1/n sum_t lse_t^2
//   d balance / d scores[t,e] = E / (n^2 K) p_te (c_e - sum_j p_tj c_j)
//   d z / d scores[t,e]       = 2/n lse_t p_te
// c is a count and has no gradient. The kept gates g = softmax(scores[idx]) add
//   sum_{k: idx[t,k] = e} g_k (dg_k - sum_j g_j dg_j).
//
// A token's E scores sit in L lanes, V x C to a lane, so that a wave reads
// 64 / L whole rows at once and a row's maximum and sums are lane exchanges; L and
// V follow from E alone (V = 4 where rows start on 4 elements). Sums over the
// tokens stay in each lane's registers, meet in LDS in a fixed order, and, with
// more than one block, in one row of the workspace per block, which a second
// launch of one block adds up in order. The backward pass recomputes p from the
// scores, which costs one read of them and saves a written and read copy.
//
// 65536 tokens of 128 fp32 scores, K = 8: forward 11 us and 4.4 for the last launch,
// backward (bf16 gradients) 21: 3.3 and 2.7 TB/s. The backward is bound by its vector
// instructions, about 140 a token of a wave, most of them the exponentials', the
// conversions' and the lane exchanges'; 64 tokens of 8 experts take 4.7 and 4.4 us,
// one block's latency.
#include "rows.h"

namespace moe {
namespace {

constexpr int kLossThreads = 1024;
constexpr int kLossWaves = kLossThreads / kWave;
constexpr int kLossTokens = 4;    // of a lane group, their loads in flight together
constexpr int kLossBlocks = 256;  // at most, of the forward pass: rows of partial sums

// The scores of one token in this lane: c-th group of V from expert (c * L + l) * V.
template <typename T, int V, int L, int C>
struct Row {
  static constexpr int kN = V * C;
  float v[kN];
  __device__ __forceinline__ int expert(int l, int i) const { return (i / V * L + l) * V + i % V; }
  __device__ __forceinline__ void load(const T* __restrict__ row, int l, int E) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * L + l) * V;
      if (e < E) {  // V > 1: E is a multiple of V
        struct __attribute__((aligned(V * sizeof(T)))) Quad { T x[V]; };
        const Quad q = *reinterpret_cast<const Quad*>(row + e);
#pragma unroll
        for (int i = 0; i < V; ++i) v[c * V + i] = to_f32(q.x[i]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[c * V + i] = -INFINITY;
      }
    }
  }
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = -INFINITY;
  }
  // v becomes exp(v - max); their sum and lse. False for a row of -inf alone (a
  // NaN is no such row: it reaches the sum, which is then not 0).
  __device__ __forceinline__ bool exps(float& sum, float& lse) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kN; ++i) m = fmaxf(m, v[i]);
    m = lanes_max<L>(m);
    const float base = m > -INFINITY ? m : 0.f;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      v[i] = __expf(v[i] - base);  // off by |v - base| steps of 2^-24 and one more (65536 x 128: 36 us both ways, expf 41)
      s += v[i];
    }
    sum = lanes_sum<L>(s);
    lse = base + logf(sum);
    return sum != 0.f;
  }
};

// The last step, by one block: probs and counts of the experts from n rows of
// partial sums (their own row pitch E), the losses from them.
__device__ __forceinline__ void finish_losses(const float* psum, const int* cnt, const float* zsum, const int* live,
                                              int rows, int E, int K, int32_t* __restrict__ counts,
                                              int32_t* __restrict__ tokens, float* __restrict__ probs,
                                              float* __restrict__ loss, float* s_f, int* s_i) {
  // thread (e, part): part of the rows' sums of expert e
  const int tid = threadIdx.x;
  const int parts = min(min(kLossThreads / E, 16), rows);
  const int e = tid % E, part = tid / E;
  if (part < parts) {
    float ps = 0.f;
    int cs = 0;
#pragma unroll 16
    for (int r = part; r < rows; r += parts) {
      ps += psum[(int64_t)r * E + e];
      cs += cnt[(int64_t)r * E + e];
    }
    s_f[part * E + e] = ps;
    s_i[part * E + e] = cs;
  }
  __shared__ float s_z, s_b[kLossWaves];
  __shared__ int s_n;
  if (tid < kWave) {
    float z = 0.f;
    int n = 0;
    for (int r = tid; r < rows; r += kWave) {
      z += zsum[r];
      n += live[r];
    }
    z = lanes_sum<kWave>(z);
    for (int off = 1; off < kWave; off <<= 1) n += __shfl_xor(n, off, kWave);
    if (tid == 0) {
      s_z = z;
      s_n = n;
    }
  }
  __syncthreads();
  float term = 0.f;
  const float per = s_n > 0 ? 1.f / (float)s_n : 0.f;
  if (tid < E) {
    float pe = 0.f;
    int ce = 0;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      pe += s_f[p * E + tid];
      ce += s_i[p * E + tid];
    }
    pe *= per;
    counts[tid] = ce;
    probs[tid] = pe;
    term = (float)ce * pe;
  }
  term = lanes_sum<kWave>(term);
  if ((tid & (kWave - 1)) == 0) s_b[tid / kWave] = term;
  __syncthreads();
  if (tid == 0) {
    float b = 0.f;
    for (int i = 0; i < kLossWaves; ++i) b += s_b[i];
    tokens[0] = s_n;
    loss[0] = b * per * (float)E / (float)K;
    loss[1] = s_z * per;
  }
}

// Block b takes tokens [b * chunk, (b + 1) * chunk).
template <typename T, int V, int L, int C>
__global__ __launch_bounds__(kLossThreads) void loss_kernel(const T* __restrict__ scores,
                                                            const int32_t* __restrict__ idx,
                                                            const uint8_t* __restrict__ mask, int T_, int E, int K,
                                                            int chunk, float* __restrict__ ws,
                                                            int32_t* __restrict__ counts, int32_t* __restrict__ tokens,
                                                            float* __restrict__ probs, float* __restrict__ loss) {
  constexpr int kPer = kWave / L;  // tokens of a wave at a time
  constexpr int U = kLossTokens;
  constexpr int kStep = kLossWaves * kPer;
  __shared__ float s_p[kLossWaves * 256];
  __shared__ int s_c[kLossThreads];  // 256 counts; finish_losses' partial counts
  __shared__ float s_zw[kLossWaves];
  __shared__ int s_nw[kLossWaves];
  const int tid = threadIdx.x, w = tid / kWave, lane = tid % kWave, l = lane % L;
  for (int i = tid; i < 256; i += kLossThreads) s_c[i] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * chunk, t1 = min(T_, t0 + chunk);
  typedef Row<T, V, L, C> R;
  float acc[R::kN];
#pragma unroll
  for (int i = 0; i < R::kN; ++i) acc[i] = 0.f;
  float zacc = 0.f;
  int nacc = 0;
  for (int tb = t0 + w * kPer + lane / L; tb - lane / L < t1; tb += U * kStep) {
    R r[U];
    bool on[U];
    int id[U];  // one chosen expert to a lane, where there are lanes enough
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = min(tb + u * kStep, t1 - 1);  // a token past the last reads the last again
      r[u].load(scores + (int64_t)t * E, l, E);
      if (L >= 8) id[u] = idx[(int64_t)t * K + min(l, K - 1)];
      on[u] = mask == nullptr || mask[t] != 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u * kStep;
      float sum, lse;
      const bool live = r[u].exps(sum, lse) && on[u] && t < t1;
      if (live) {
        const float inv = 1.f / sum;
#pragma unroll
        for (int i = 0; i < R::kN; ++i) acc[i] = fmaf(r[u].v[i], inv, acc[i]);
        if (l == 0) {
          zacc = fmaf(lse, lse, zacc);
          ++nacc;
        }
        // whole numbers: any order
        if (L >= 8) {
          if (l < K && id[u] >= 0 && id[u] < E) atomicAdd(&s_c[id[u]], 1);
        } else {
          for (int k = l; k < K; k += L) {
            const int e = idx[(int64_t)t * K + k];
            if (e >= 0 && e < E) atomicAdd(&s_c[e], 1);
          }
        }
      }
    }
  }
  // the wave's groups of lanes, in order of halves, then the waves in order
#pragma unroll
  for (int i = 0; i < R::kN; ++i) {
    float a = acc[i];
    for (int off = L; off < kWave; off <<= 1) a += __shfl_xor(a, off, kWave);
    const int e = (i / V * L + l) * V + i % V;
    if (lane < L && e < E) s_p[w * 256 + e] = a;
  }
  for (int off = 1; off < kWave; off <<= 1) {
    zacc += __shfl_xor(zacc, off, kWave);
    nacc += __shfl_xor(nacc, off, kWave);
  }
  if (lane == 0) {
    s_zw[w] = zacc;
    s_nw[w] = nacc;
  }
  __syncthreads();
  float ps = 0.f;
  if (tid < E)
    for (int i = 0; i < kLossWaves; ++i) ps += s_p[i * 256 + tid];
  float z = 0.f;
  int n = 0;
  for (int i = 0; i < kLossWaves; ++i) {
    z += s_zw[i];
    n += s_nw[i];
  }
  const int ce = tid < E ? s_c[tid] : 0;
  __syncthreads();
  if (gridDim.x == 1) {
    if (tid < E) {
      s_p[kLossThreads + tid] = ps;  // one row of partial sums, behind finish_losses' own
      s_p[kLossThreads + 256 + tid] = __int_as_float(ce);
    }
    if (tid == 0) {
      s_zw[0] = z;
      s_nw[0] = n;
    }
    __syncthreads();
    finish_losses(s_p + kLossThreads, reinterpret_cast<const int*>(s_p + kLossThreads + 256), s_zw, s_nw, 1, E, K,
                  counts, tokens, probs, loss, s_p, s_c);
    return;
  }
  float* wp = ws + (int64_t)blockIdx.x * E;
  int* wc = reinterpret_cast<int*>(ws + (int64_t)gridDim.x * E) + (int64_t)blockIdx.x * E;
  float* wz = ws + (int64_t)gridDim.x * 2 * E + blockIdx.x;
  int* wn = reinterpret_cast<int*>(ws + (int64_t)gridDim.x * (2 * E + 1)) + blockIdx.x;
  if (tid < E) {
    wp[tid] = ps;
    wc[tid] = ce;
  }
  if (tid == 0) {
    *wz = z;
    *wn = n;
  }
}

__global__ __launch_bounds__(kLossThreads) void loss_finish_kernel(const float* __restrict__ ws, int rows, int E,
                                                                   int K, int32_t* __restrict__ counts,
                                                                   int32_t* __restrict__ tokens,
                                                                   float* __restrict__ probs,
                                                                   float* __restrict__ loss) {
  __shared__ float s_f[kLossThreads];
  __shared__ int s_i[kLossThreads];
  finish_losses(ws, reinterpret_cast<const int*>(ws + (int64_t)rows * E), ws + (int64_t)rows * 2 * E,
                reinterpret_cast<const int*>(ws + (int64_t)rows * (2 * E + 1)), rows, E, K, counts, tokens, probs,
                loss, s_f, s_i);
}

// Lane k of every 16, in all of them.
template <int K0>
__device__ __forceinline__ int row_bcast(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x150 + K0, 0xf, 0xf, true);  // row_newbcast
}

template <int K0, int N>
struct AddSlots {
  template <typename E>
  static __device__ __forceinline__ void run(int slot, float part, int K, float (&d)[N], E expert) {
    if (K0 < K) {
      const int e = row_bcast<K0>(slot);
      const float p = __int_as_float(row_bcast<K0>(__float_as_int(part)));
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] += expert(i) == e ? p : 0.f;
    }
    if constexpr (K0 < 7) AddSlots<K0 + 1, N>::run(slot, part, K, d, expert);
  }
};

template <typename T, typename O, int V, int L, int C>
__global__ __launch_bounds__(256) void loss_bwd_kernel(const T* __restrict__ scores, const int32_t* __restrict__ idx,
                                                       const uint8_t* __restrict__ mask,
                                                       const int32_t* __restrict__ counts,
                                                       const int32_t* __restrict__ tokens,
                                                       const float* __restrict__ dloss,
                                                       const float* __restrict__ gate,
                                                       const float* __restrict__ dgate, int T_, int E, int K,
                                                       O* __restrict__ out) {
  constexpr int kPer = kWave / L;
  constexpr int U = kLossTokens;
  const int w = threadIdx.x / kWave, lane = threadIdx.x % kWave, l = lane % L;
  typedef Row<T, V, L, C> R;
  float c[R::kN];
  float cb = 0.f, cz = 0.f;
  if (dloss != nullptr) {
    const int n = tokens[0];
    const float per = n > 0 ? 1.f / (float)n : 0.f;
    cb = dloss[0] * per * per * (float)E / (float)K;
    cz = dloss[1] * 2.f * per;
  }
#pragma unroll
  for (int i = 0; i < R::kN; ++i) {
    const int e = (i / V * L + l) * V + i % V;
    c[i] = dloss != nullptr && e < E ? (float)counts[e] : 0.f;
  }
  const int64_t first = ((int64_t)blockIdx.x * 4 + w) * kPer * U + lane / L;
  R r[U];
  bool on[U];
  int slot[U];  // L >= 16: slot k of the token in lane k of every 16
  float g[U], dg[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = min(first + u * kPer, (int64_t)T_ - 1);  // a token past the last reads the last again
    on[u] = false;
    if (dloss != nullptr) {
      r[u].load(scores + t * E, l, E);
      on[u] = mask == nullptr || mask[t] != 0;
    } else {
      r[u].none();
    }
    if (L >= 16 && dgate != nullptr) {
      const int64_t at = t * K + min(lane & 15, K - 1);
      slot[u] = idx[at];
      g[u] = gate[at];
      dg[u] = dgate[at];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = first + u * kPer;
    const bool in = t < T_;
    float sum, lse, d[R::kN];
    const bool live = r[u].exps(sum, lse) && on[u] && in;
    const float inv = live ? 1.f / sum : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < R::kN; ++i) {
      d[i] = live ? r[u].v[i] * inv : 0.f;
      dot = fmaf(d[i], c[i], dot);
    }
    dot = lanes_sum<L>(dot);
    // a token without a part has none of a gradient that is no number either
    const float bt = live ? cb : 0.f, zt = live ? cz * lse : 0.f;
#pragma unroll
    for (int i = 0; i < R::kN; ++i) d[i] *= fmaf(bt, c[i] - dot, zt);
    if (dgate != nullptr) {
      const auto expert = [&](int i) { return (i / V * L + l) * V + i % V; };
      if (L >= 16) {
        const bool mine = (lane & 15) < K && slot[u] >= 0 && slot[u] < E;
        const float s = lanes_sum<16>(mine ? g[u] * dg[u] : 0.f);
        AddSlots<0, R::kN>::run(slot[u], g[u] * (dg[u] - s), K, d, expert);
      } else if (in) {
        float s = 0.f;
        for (int k = 0; k < K; ++k) {
          const int e = idx[t * K + k];
          if (e >= 0 && e < E) s = fmaf(gate[t * K + k], dgate[t * K + k], s);
        }
        for (int k = 0; k < K; ++k) {
          const int e = idx[t * K + k];
          if (e < 0 || e >= E) continue;
          const float p = gate[t * K + k] * (dgate[t * K + k] - s);
#pragma unroll
          for (int i = 0; i < R::kN; ++i) d[i] += expert(i) == e ? p : 0.f;
        }
      }
    }
    if (!in) continue;
    O* row = out + t * E;
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int e = (q * L + l) * V;
      if (e >= E) continue;
      struct __attribute__((aligned(V * sizeof(O)))) Quad { O x[V]; } o;
#pragma unroll
      for (int i = 0; i < V; ++i) from_f32(d[q * V + i], o.x[i]);
      *reinterpret_cast<Quad*>(row + e) = o;
    }
  }
}

// Calls f(V, L, C) with E's layout as compile-time numbers.
template <typename F>
moe_status with_layout(int E, F f) {
#define MOE_LAYOUT(V, L, C) return f(std::integral_constant<int, V>{}, std::integral_constant<int, L>{}, std::integral_constant<int, C>{})
  if (E % 4 == 0) {
    const int q = E / 4;
    if (q <= 1) MOE_LAYOUT(4, 1, 1);
    if (q <= 2) MOE_LAYOUT(4, 2, 1);
    if (q <= 4) MOE_LAYOUT(4, 4, 1);
    if (q <= 8) MOE_LAYOUT(4, 8, 1);
    if (q <= 16) MOE_LAYOUT(4, 16, 1);
    if (q <= 32) MOE_LAYOUT(4, 32, 1);
    MOE_LAYOUT(4, 64, 1);
  }
  if (E <= 2) MOE_LAYOUT(1, 2, 1);
  if (E <= 8) MOE_LAYOUT(1, 8, 1);
  if (E <= 16) MOE_LAYOUT(1, 16, 1);
  if (E <= 32) MOE_LAYOUT(1, 16, 2);
  if (E <= 64) MOE_LAYOUT(1, 16, 4);
  if (E <= 128) MOE_LAYOUT(1, 32, 4);
  MOE_LAYOUT(1, 64, 4);
#undef MOE_LAYOUT
}

// Tokens per block of the forward pass, and the blocks: one block takes up to two
// rounds of its waves alone, one launch instead of two (512 x 64: 8.5 us, in two launches
// 7.9 and another launch's host time; four rounds, 1024 x 64: 13.2 and 8.0).
struct LossPlan {
  int chunk, blocks;
};
LossPlan loss_plan(int T, int E) {
  int step = 0;
  with_layout(E, [&](auto v, auto l, auto c) {
    step = kLossWaves * (kWave / l) * kLossTokens;
    return MOE_OK;
  });
  if (T <= 2 * step) return {T > 0 ? T : 1, 1};
  const int64_t per = cdiv64(cdiv64(T, kLossBlocks), step) * step;
  return {(int)per, (int)cdiv64(T, per)};
}

}  // namespace

size_t router_loss_ws_bytes(int T, int E) {
  const LossPlan p = loss_plan(T, E);
  return p.blocks > 1 ? (size_t)p.blocks * (2 * E + 2) * 4 : 0;
}

moe_status launch_router_loss(const void* scores, moe_dtype dt, const int32_t* idx, const uint8_t* mask, int T, int E,
                              int K, int32_t* counts, int32_t* tokens, float* probs, float* loss, void* ws,
                              hipStream_t s) {
  const LossPlan p = loss_plan(T, E);
  with_layout(E, [&](auto v, auto l, auto c) {
    const dim3 grid(p.blocks), block(kLossThreads);
    if (dt == MOE_F32)
      hipLaunchKernelGGL((loss_kernel<float, v(), l(), c()>), grid, block, 0, s, (const float*)scores, idx, mask, T, E,
                         K, p.chunk, (float*)ws, counts, tokens, probs, loss);
    else
      hipLaunchKernelGGL((loss_kernel<bf16_t, v(), l(), c()>), grid, block, 0, s, (const bf16_t*)scores, idx, mask, T,
                         E, K, p.chunk, (float*)ws, counts, tokens, probs, loss);
    return MOE_OK;
  });
  if (p.blocks > 1)
    hipLaunchKernelGGL(loss_finish_kernel, dim3(1), dim3(kLossThreads), 0, s, (const float*)ws, p.blocks, E, K, counts,
                       tokens, probs, loss);
  return launch_status();
}

moe_status launch_router_loss_bwd(const void* scores, moe_dtype dt, const int32_t* idx, const uint8_t* mask,
                                  const int32_t* counts, const int32_t* tokens, const float* dloss, const float* gate,
                                  const float* dgate, int T, int E, int K, void* out, moe_dtype out_dt,
                                  hipStream_t s) {
  if (T == 0) return MOE_OK;
  with_layout(E, [&](auto v, auto l, auto c) {
    constexpr int per = 4 * (kWave / l()) * kLossTokens;
    const dim3 grid((unsigned)cdiv64(T, per)), block(256);
    const auto go = [&](auto in, auto o) {
      typedef decltype(in) TI;
      typedef decltype(o) TO;
      hipLaunchKernelGGL((loss_bwd_kernel<TI, TO, v(), l(), c()>), grid, block, 0, s, (const TI*)scores, idx, mask,
                         counts, tokens, dloss, gate, dgate, T, E, K, (TO*)out);
    };
    if (dt == MOE_F32 && out_dt == MOE_F32) go(float(), float());
    else if (dt == MOE_F32) go(float(), bf16_t());
    else if (out_dt == MOE_F32) go(bf16_t(), float());
    else go(bf16_t(), bf16_t());
    return MOE_OK;
  });
  return launch_status();
}

}  // namespace moe
