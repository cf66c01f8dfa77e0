// norm.hip — the norms after and before a block, with its gate and residual scale:
//   u = post(z),  r' = alpha r + beta g u,  h = pre(r')
// post and pre: n w + b with n = (x - m) / sqrt(mean (x - m)^2 + eps), m the row's
// mean (layer norm) or 0 (RMS norm). The gate g is one number per channel, or per
// token, or 1. Backwards, with D = dr' + pre's gradient of dh:
//   pre's gradient of d at x:  rstd (e - n mean(e n) - mean(e)), e = d w (the last
//                              mean for layer norms only)
//   dr = alpha D,  du = beta g D,  dz = post's gradient of du (du without post)
//   dw_pre = sum_t dh n', db_pre = sum_t dh, and with S1 = sum_t c_t D n, S0 = sum_t c_t D
//   (c_t = beta, times the token's gate): dw_post = g S1, db_post = g S0, a channel's
//   dgate = w_post S1 + b_post S0, a token's dgate = beta sum_n D u.
//
// HBM-bound: a row is read once into registers, 8 values per lane and access, by
// one wave up to one block; every mean is a lane exchange (and an LDS step between
// waves); means of a layer norm come first and squares of differences second, so
// that a large mean costs no precision.
//
// 8192 x 7168 bf16 (RMS norms, z, r, r' and h): 97 us, 4.9 TB/s, the rate of a copy;
// 777 x 1501 (rows on no boundary): 7.4 us; one row of 4096: 3.2 us.
#include "norm.h"

namespace moe {
namespace {

// W waves to a row, C accesses of 8 values to a lane.
template <typename TZ, typename TR, int W, int C, int MODE>
__global__ __launch_bounds__(W > 4 ? W * kWave : 256) void norm_kernel(NormCall c) {
  constexpr int kRows = W > 4 ? 1 : 4 / W;  // rows of a block
  typedef RowVec<TZ, kNV, MODE, MODE == kWhole> Z;
  typedef RowVec<TR, kNV, MODE, MODE == kWhole> R;
  __shared__ __attribute__((aligned(16))) float s[kRows][2][W][4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wr = wave % W, sub = wave / W;
  const int64_t t = (int64_t)blockIdx.x * kRows + sub;
  const bool in = t < c.T;
  if (W == 1 && !in) return;  // no barrier to reach
  const int N = c.N;
  const int64_t at = (in ? t : 0) * N;  // row 0 stands in for a row past the last
  const float per = 1.f / (float)N;
  const bool layer = c.kind == MOE_NORM_LAYER;
  int slot = 0;
  const auto col = [&](int q) { return ((q * W + wr) * kWave + (int)threadIdx.x % kWave) * kNV; };
  const auto on = [&](int q, int i) { return MODE == kWhole ? col(q) < N : col(q) + i < N; };
  float x[C][kNV];
  // mean and 1 / size of the row in x
  const auto stats = [&](float& mean, float& rstd) {
    float m[1] = {0.f};
    mean = 0.f;
    if (layer) {
#pragma unroll
      for (int q = 0; q < C; ++q)
#pragma unroll
        for (int i = 0; i < kNV; ++i) m[0] += x[q][i];
      row_sums<W, 1>(m, s[sub], wr, slot);
      mean = m[0] * per;
    }
    m[0] = 0.f;
#pragma unroll
    for (int q = 0; q < C; ++q)
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const float d = layer && !on(q, i) ? 0.f : x[q][i] - mean;
        m[0] = fmaf(d, d, m[0]);
      }
    row_sums<W, 1>(m, s[sub], wr, slot);
    rstd = 1.f / sqrtf(m[0] * per + c.eps);
  };
  float mean, rstd;
  if (c.z != nullptr) {
    Z z[C];
    R r[C];
#pragma unroll
    for (int q = 0; q < C; ++q) z[q].load((const TZ*)c.z + at, col(q), N);
    if (c.r != nullptr)
#pragma unroll
      for (int q = 0; q < C; ++q) r[q].load((const TR*)c.r + at, col(q), N);
    const void* channel = c.gate_mode == MOE_GATE_CHANNEL ? c.gate : nullptr;
#pragma unroll
    for (int q = 0; q < C; ++q) z[q].get(x[q], col(q), N);
    mean = 0.f;
    rstd = 1.f;
    if (c.post) stats(mean, rstd);
    float ct = c.beta;
    if (c.gate_mode == MOE_GATE_TOKEN && in) ct *= load_w1(c.gate, c.w_f32, t);
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int j = col(q);
      float w[kNV], b[kNV], g[kNV], v[kNV], o[kNV];
      load_w<MODE>(c.w_post, c.w_f32, j, N, w, 1.f);
      load_w<MODE>(c.b_post, c.w_f32, j, N, b, 0.f);
      load_w<MODE>(channel, c.w_f32, j, N, g, 1.f);
      if (c.r != nullptr) r[q].get(v, j, N);
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        o[i] = ct * g[i] * fmaf((x[q][i] - mean) * rstd, w[i], b[i]);
        if (c.r != nullptr) o[i] = fmaf(c.alpha, v[i], o[i]);
        if (!on(q, i)) o[i] = 0.f;
      }
      R out;
      out.put(o);
#pragma unroll
      for (int i = 0; i < kNV; ++i) x[q][i] = out.at(i);  // h is the norm of r' as it is stored
      if (c.r_out != nullptr && in) out.store((TR*)c.r_out + at, j, N);
    }
  } else {
    R r[C];
#pragma unroll
    for (int q = 0; q < C; ++q) r[q].load((const TR*)c.r + at, col(q), N);
#pragma unroll
    for (int q = 0; q < C; ++q) r[q].get(x[q], col(q), N);
  }
  if (c.h == nullptr) return;
  stats(mean, rstd);
#pragma unroll
  for (int q = 0; q < C; ++q) {
    const int j = col(q);
    float w[kNV], b[kNV], o[kNV];
    load_w<MODE>(c.w_pre, c.w_f32, j, N, w, 1.f);
    load_w<MODE>(c.b_pre, c.w_f32, j, N, b, 0.f);
#pragma unroll
    for (int i = 0; i < kNV; ++i) o[i] = fmaf((x[q][i] - mean) * rstd, w[i], b[i]);
    Z out;
    out.put(o);
    if (in) out.store((TZ*)c.h + at, j, N);
  }
}

// Waves per row and accesses per lane: one access of each array to a lane while 16
// waves hold the row (8192 x 4096: 52 us, against 63 with one wave of eight; one row of
// 4096: 4 us against 8), but two where many rows are short (8192 x 1024: 15 us against
// 17; 2048 wide both take the same).
struct NormPlan {
  int W, C;
};
NormPlan norm_plan(int64_t T, int N) {
  const int need = (N + kNV * kWave - 1) / (kNV * kWave);  // accesses of one wave
  const int per = T >= 2048 && need > 1 && need <= 3 ? 2 : 1;
  NormPlan p{1, 1};
  while (p.W < 16 && p.W * per < need) p.W *= 2;
  while (p.W * p.C < need) p.C *= 2;
  return p;
}

// A launch has fewer than 2^32 threads (with more, nothing runs and no error is reported):
// more rows than that take another (8.4 million rows of 2049 to 4096).
template <typename TZ, typename TR, int W, int C>
void go_norm(NormCall c, hipStream_t s) {
  constexpr int rows = W > 4 ? 1 : 4 / W, threads = W > 4 ? W * kWave : 256;
  constexpr int64_t most = 0xffffffffll / threads * rows;
  const auto from = [](const void*& p, int64_t bytes) {
    if (p != nullptr) p = (const unsigned char*)p + bytes;
  };
  const auto into = [](void*& p, int64_t bytes) {
    if (p != nullptr) p = (unsigned char*)p + bytes;
  };
  for (int64_t left = c.T; left > 0; left -= most) {
    c.T = (int)(left < most ? left : most);
    with_mode(row_mode(c.N, kNV), [&](auto mode) {
      if constexpr (mode() != kNarrow || (W == 1 && C == 1))
        hipLaunchKernelGGL((norm_kernel<TZ, TR, W, C, mode()>), dim3((unsigned)cdiv64(c.T, rows)), dim3(threads), 0, s, c);
    });
    from(c.z, most * c.N * sizeof(TZ));
    from(c.r, most * c.N * sizeof(TR));
    if (c.gate_mode == MOE_GATE_TOKEN) from(c.gate, most * (c.w_f32 ? 4 : 2));
    into(c.r_out, most * c.N * sizeof(TR));
    into(c.h, most * c.N * sizeof(TZ));
  }
}

template <typename TZ, typename TR>
void pick_norm(const NormCall& c, hipStream_t s) {
  const NormPlan p = norm_plan(c.T, c.N);
#define MOE_NORM(w, n) if (p.W == w && p.C == n) return go_norm<TZ, TR, w, n>(c, s)
  MOE_NORM(1, 1); MOE_NORM(2, 1); MOE_NORM(4, 1); MOE_NORM(8, 1); MOE_NORM(16, 1);
  MOE_NORM(1, 2); MOE_NORM(2, 2); MOE_NORM(16, 2); MOE_NORM(16, 4); MOE_NORM(16, 8);
#undef MOE_NORM
}

}  // namespace

moe_status launch_norm(const NormCall& c, moe_dtype dt, moe_dtype r_dt, hipStream_t s) {
  if (c.T == 0) return MOE_OK;
  if (dt == MOE_F32) pick_norm<float, float>(c, s);
  else if (r_dt == MOE_F32) pick_norm<bf16_t, float>(c, s);
  else pick_norm<bf16_t, bf16_t>(c, s);
  return launch_status();
}

}  // namespace moe
