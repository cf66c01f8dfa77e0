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
#include "rows.h"

namespace moe {
namespace {

constexpr int kNV = 8;  // values per lane and access

// Values of a norm's weight or a gate, in binary32 or bf16 (the same in all lanes).
__device__ __forceinline__ void load_w(const void* w, bool f32, int j, int n, float (&o)[kNV], float none) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < kNV; ++i) o[i] = none;
  } else if (f32) {
    const Vec<float, kNV> v = load_vec<float, kNV>((const float*)w, j, n);
#pragma unroll
    for (int i = 0; i < kNV; ++i) o[i] = v.v[i];
  } else {
    const Vec<bf16_t, kNV> v = load_vec<bf16_t, kNV>((const bf16_t*)w, j, n);
#pragma unroll
    for (int i = 0; i < kNV; ++i) o[i] = bf16_to_f32(v.v[i]);
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
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) a += s[slot][i][q];
      v[q] = a;
    }
    slot ^= 1;
  }
}

// W waves to a row, C accesses of 8 values to a lane.
template <typename TZ, typename TR, int W, int C>
__global__ __launch_bounds__(W > 4 ? W * kWave : 256) void norm_kernel(NormCall c) {
  constexpr int kRows = W > 4 ? 1 : 4 / W;  // rows of a block
  __shared__ float s[kRows][2][W][4];
  const int wave = threadIdx.x / kWave, wr = wave % W, sub = wave / W;
  const int lane = wr * kWave + threadIdx.x % kWave;  // of the row
  const int64_t t = (int64_t)blockIdx.x * kRows + sub;
  const bool in = t < c.T;
  if (W == 1 && !in) return;  // no barrier to reach
  const int N = c.N;
  const int64_t at = (in ? t : 0) * N;
  const float per = 1.f / (float)N;
  const bool layer = c.kind == MOE_NORM_LAYER;
  int slot = 0;
  const TZ* z = (const TZ*)c.z + at;
  const TR* r = (const TR*)c.r + at;
  float x[C][kNV];
  if (c.z != nullptr) {
    Vec<TZ, kNV> zv[C];
    Vec<TR, kNV> rv[C];
#pragma unroll
    for (int q = 0; q < C; ++q) zv[q] = load_vec<TZ, kNV>(z, (q * W * kWave + lane) * kNV, N);
    if (c.r != nullptr)
#pragma unroll
      for (int q = 0; q < C; ++q) rv[q] = load_vec<TR, kNV>(r, (q * W * kWave + lane) * kNV, N);
#pragma unroll
    for (int q = 0; q < C; ++q)
#pragma unroll
      for (int i = 0; i < kNV; ++i) x[q][i] = to_f32(zv[q].v[i]);
    float mean = 0.f, rstd = 1.f;
    if (c.post) {
      float m[1] = {0.f};
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
          const float d = (q * W * kWave + lane) * kNV + i < N ? x[q][i] - mean : 0.f;
          m[0] = fmaf(d, d, m[0]);
        }
      row_sums<W, 1>(m, s[sub], wr, slot);
      rstd = 1.f / sqrtf(m[0] * per + c.eps);
    }
    float ct = c.beta;
    if (c.gate_mode == MOE_GATE_TOKEN && in) ct *= load_w1(c.gate, c.w_f32, t);
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int j = (q * W * kWave + lane) * kNV;
      float w[kNV], b[kNV], g[kNV];
      load_w(c.w_post, c.w_f32, j, N, w, 1.f);
      load_w(c.b_post, c.w_f32, j, N, b, 0.f);
      load_w(c.gate_mode == MOE_GATE_CHANNEL ? c.gate : nullptr, c.w_f32, j, N, g, 1.f);
      Vec<TR, kNV> o;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const float u = fmaf((x[q][i] - mean) * rstd, w[i], b[i]);
        float v = ct * g[i] * u;
        if (c.r != nullptr) v = fmaf(c.alpha, to_f32(rv[q].v[i]), v);
        from_f32(v, o.v[i]);
        x[q][i] = to_f32(o.v[i]);  // h is the norm of r' as it is stored
      }
      if (c.r_out != nullptr && in) store_vec<TR, kNV>((TR*)c.r_out + at, j, N, o);
    }
  } else {
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const Vec<TR, kNV> v = load_vec<TR, kNV>(r, (q * W * kWave + lane) * kNV, N);
#pragma unroll
      for (int i = 0; i < kNV; ++i) x[q][i] = to_f32(v.v[i]);
    }
  }
  if (c.h == nullptr) return;
  float mean = 0.f, m[1] = {0.f};
  if (layer) {
#pragma unroll
    for (int q = 0; q < C; ++q)
#pragma unroll
      for (int i = 0; i < kNV; ++i) m[0] += (q * W * kWave + lane) * kNV + i < N ? x[q][i] : 0.f;
    row_sums<W, 1>(m, s[sub], wr, slot);
    mean = m[0] * per;
  }
  m[0] = 0.f;
#pragma unroll
  for (int q = 0; q < C; ++q)
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const float d = (q * W * kWave + lane) * kNV + i < N ? x[q][i] - mean : 0.f;
      m[0] = fmaf(d, d, m[0]);
    }
  row_sums<W, 1>(m, s[sub], wr, slot);
  const float rstd = 1.f / sqrtf(m[0] * per + c.eps);
#pragma unroll
  for (int q = 0; q < C; ++q) {
    const int j = (q * W * kWave + lane) * kNV;
    float w[kNV], b[kNV];
    load_w(c.w_pre, c.w_f32, j, N, w, 1.f);
    load_w(c.b_pre, c.w_f32, j, N, b, 0.f);
    Vec<TZ, kNV> o;
#pragma unroll
    for (int i = 0; i < kNV; ++i) from_f32(fmaf((x[q][i] - mean) * rstd, w[i], b[i]), o.v[i]);
    if (in) store_vec<TZ, kNV>((TZ*)c.h + at, j, N, o);
  }
}

// ------------------------------------------------------------------ backward

// Sums over a block's rows go to its four rows of the workspace (dh n', dh, S1, S0 of
// kNormSums), N apart; the finishing launch adds the blocks in order.
constexpr int kNormSums = 4;

template <typename TZ, typename TR, bool LAYER, int W, int C>
__global__ __launch_bounds__(W > 4 ? W * kWave : 256) void norm_bwd_kernel(NormBwdCall c) {
  constexpr int kRows = W > 4 ? 1 : 4 / W;
  __shared__ float s[kRows][2][W][4];
  const int wave = threadIdx.x / kWave, wr = wave % W, sub = wave / W;
  const int lane = wr * kWave + threadIdx.x % kWave;
  const int N = c.N;
  const float per = 1.f / (float)N;
  float d1[C][kNV], d0[C][kNV], s1[C][kNV], s0[C][kNV];
#pragma unroll
  for (int q = 0; q < C; ++q)
#pragma unroll
    for (int i = 0; i < kNV; ++i) d1[q][i] = d0[q][i] = s1[q][i] = s0[q][i] = 0.f;
  int slot = 0;
  // the rows of a block are walked by all of its waves together: the barriers match
  for (int64_t tb = (int64_t)blockIdx.x * kRows; tb < c.T; tb += (int64_t)gridDim.x * kRows) {
    const int64_t t = tb + sub;
    const bool in = t < c.T;
    const int64_t at = (in ? t : 0) * N;
    float x[C][kNV], dd[C][kNV], z[C][kNV], dr[C][kNV];
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int j = (q * W * kWave + lane) * kNV, n = in ? N : 0;
      const Vec<TR, kNV> xv = c.dh ? load_vec<TR, kNV>((const TR*)c.r_out + at, j, n) : Vec<TR, kNV>{};
      const Vec<TZ, kNV> dv = c.dh ? load_vec<TZ, kNV>((const TZ*)c.dh + at, j, n) : Vec<TZ, kNV>{};
      const Vec<TZ, kNV> zv = c.z ? load_vec<TZ, kNV>((const TZ*)c.z + at, j, n) : Vec<TZ, kNV>{};
      const Vec<TR, kNV> rv = c.dr_out ? load_vec<TR, kNV>((const TR*)c.dr_out + at, j, n) : Vec<TR, kNV>{};
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        x[q][i] = to_f32(xv.v[i]);
        dd[q][i] = to_f32(dv.v[i]);
        z[q][i] = to_f32(zv.v[i]);
        dr[q][i] = to_f32(rv.v[i]);
      }
    }
    float mx = 0.f, mz = 0.f;
    if (LAYER) {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int q = 0; q < C; ++q)
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          m[0] += x[q][i];
          m[1] += z[q][i];
        }
      row_sums<W, 2>(m, s[sub], wr, slot);
      mx = m[0] * per;
      mz = c.post ? m[1] * per : 0.f;
    }
    // squares of the two rows, and what pre's gradient needs of e = dh w
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int j = (q * W * kWave + lane) * kNV;
      float w[kNV];
      load_w(c.w_pre, c.w_f32, j, N, w, 1.f);
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const bool on = j + i < N;
        x[q][i] = on ? x[q][i] - mx : 0.f;
        z[q][i] = on ? z[q][i] - mz : 0.f;
        const float e = dd[q][i] * w[i];
        a[0] = fmaf(x[q][i], x[q][i], a[0]);
        a[1] = fmaf(z[q][i], z[q][i], a[1]);
        a[2] = fmaf(e, x[q][i], a[2]);
        a[3] += e;
      }
    }
    row_sums<W, 4>(a, s[sub], wr, slot);
    const float rx = c.dh ? 1.f / sqrtf(a[0] * per + c.eps) : 0.f;
    const float rz = c.post ? 1.f / sqrtf(a[1] * per + c.eps) : 1.f;
    const float m1 = a[2] * rx * per, m0 = LAYER ? a[3] * per : 0.f;
    float gt = 1.f;
    if (c.gate_mode == MOE_GATE_TOKEN && in) gt = load_w1(c.gate, c.w_f32, t);
    const float ct = c.beta * gt;
    float b[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int j = (q * W * kWave + lane) * kNV;
      float w[kNV], wp[kNV], bp[kNV], g[kNV];
      load_w(c.w_pre, c.w_f32, j, N, w, 1.f);
      load_w(c.w_post, c.w_f32, j, N, wp, 1.f);
      load_w(c.gate_mode == MOE_GATE_TOKEN ? c.b_post : nullptr, c.w_f32, j, N, bp, 0.f);
      load_w(c.gate_mode == MOE_GATE_CHANNEL ? c.gate : nullptr, c.w_f32, j, N, g, 1.f);
      Vec<TR, kNV> o;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const float n2 = x[q][i] * rx;
        if (c.dh != nullptr) dr[q][i] += rx * (dd[q][i] * w[i] - n2 * m1 - m0);
        from_f32(c.alpha * dr[q][i], o.v[i]);
        const float n = z[q][i] * rz;
        const float cd = ct * dr[q][i];
        if (in) {
          d1[q][i] = fmaf(dd[q][i], n2, d1[q][i]);
          s1[q][i] = fmaf(cd, n, s1[q][i]);
          if (LAYER) {
            d0[q][i] += dd[q][i];
            s0[q][i] += cd;
          }
        }
        if (j + i < N) b[2] = fmaf(dr[q][i], fmaf(n, wp[i], bp[i]), b[2]);
        z[q][i] = n;
        dr[q][i] = cd * g[i];  // du
        const float e = dr[q][i] * wp[i];
        if (j + i < N) {
          b[0] = fmaf(e, n, b[0]);
          b[1] += e;
        }
      }
      if (c.dr != nullptr && in) store_vec<TR, kNV>((TR*)c.dr + at, j, N, o);
    }
    if (c.z == nullptr) continue;
    row_sums<W, 3>(b, s[sub], wr, slot);
    if (c.gate_mode == MOE_GATE_TOKEN && c.dgate != nullptr && in && lane == 0) {
      const float dg = c.beta * b[2];
      if (c.dw_f32) ((float*)c.dgate)[t] = dg;
      else ((bf16_t*)c.dgate)[t] = f32_to_bf16(dg);
    }
    const float k1 = c.post ? b[0] * per : 0.f, k0 = LAYER && c.post ? b[1] * per : 0.f;
    if (c.dz != nullptr && in)
#pragma unroll
      for (int q = 0; q < C; ++q) {
        const int j = (q * W * kWave + lane) * kNV;
        float wp[kNV];
        load_w(c.w_post, c.w_f32, j, N, wp, 1.f);
        Vec<TZ, kNV> o;
#pragma unroll
        for (int i = 0; i < kNV; ++i) from_f32(rz * (dr[q][i] * wp[i] - z[q][i] * k1 - k0), o.v[i]);
        store_vec<TZ, kNV>((TZ*)c.dz + at, j, N, o);
      }
  }
  if (c.sums == nullptr) return;
  float* row = c.sums + ((int64_t)blockIdx.x * kRows + sub) * kNormSums * N;
#pragma unroll
  for (int q = 0; q < C; ++q) {
    const int j = (q * W * kWave + lane) * kNV;
    const auto put = [&](int which, const float (&v)[kNV]) {
      Vec<float, kNV> o;
#pragma unroll
      for (int i = 0; i < kNV; ++i) o.v[i] = v[i];
      store_vec<float, kNV>(row + (int64_t)which * N, j, N, o);
    };
    if (c.use & 1) put(0, d1[q]);
    if (c.use & 2) put(1, d0[q]);
    if (c.use & 4) put(2, s1[q]);
    if (c.use & 8) put(3, s0[q]);
  }
}

// Rows wider than the registers hold: a block of 16 waves per row, read again from
// memory (the caches) at each of its steps; the block's sums live in its rows of the
// workspace, each column touched by one lane only.
template <typename TZ, typename TR, bool LAYER>
__global__ __launch_bounds__(1024) void norm_bwd_wide_kernel(NormBwdCall c) {
  constexpr int W = 16;
  __shared__ float s[2][W][4];
  const int wr = threadIdx.x / kWave;
  const int N = c.N, step = 1024 * kNV;
  const float per = 1.f / (float)N;
  float* row = c.sums ? c.sums + (int64_t)blockIdx.x * kNormSums * N : nullptr;
  int slot = 0;
  bool first = true;
  for (int64_t t = blockIdx.x; t < c.T; t += gridDim.x, first = false) {
    const int64_t at = t * N;
    const TZ* dh = (const TZ*)c.dh + at;
    const TZ* z = (const TZ*)c.z + at;
    const TR* x = (const TR*)c.r_out + at;
    const TR* dr = (const TR*)c.dr_out + at;
    float m[2] = {0.f, 0.f};
    if (LAYER) {
      for (int j = threadIdx.x * kNV; j < N; j += step) {
        const Vec<TR, kNV> xv = c.dh ? load_vec<TR, kNV>(x, j, N) : Vec<TR, kNV>{};
        const Vec<TZ, kNV> zv = c.post ? load_vec<TZ, kNV>(z, j, N) : Vec<TZ, kNV>{};
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          m[0] += to_f32(xv.v[i]);
          m[1] += to_f32(zv.v[i]);
        }
      }
      row_sums<W, 2>(m, s, wr, slot);
    }
    const float mx = m[0] * per, mz = m[1] * per;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = threadIdx.x * kNV; j < N; j += step) {
      const Vec<TR, kNV> xv = c.dh ? load_vec<TR, kNV>(x, j, N) : Vec<TR, kNV>{};
      const Vec<TZ, kNV> dv = c.dh ? load_vec<TZ, kNV>(dh, j, N) : Vec<TZ, kNV>{};
      const Vec<TZ, kNV> zv = c.post ? load_vec<TZ, kNV>(z, j, N) : Vec<TZ, kNV>{};
      float w[kNV];
      load_w(c.w_pre, c.w_f32, j, N, w, 1.f);
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        if (j + i >= N) continue;
        const float xc = to_f32(xv.v[i]) - mx, zc = to_f32(zv.v[i]) - mz, e = to_f32(dv.v[i]) * w[i];
        a[0] = fmaf(xc, xc, a[0]);
        a[1] = fmaf(zc, zc, a[1]);
        a[2] = fmaf(e, xc, a[2]);
        a[3] += e;
      }
    }
    row_sums<W, 4>(a, s, wr, slot);
    const float rx = c.dh ? 1.f / sqrtf(a[0] * per + c.eps) : 0.f;
    const float rz = c.post ? 1.f / sqrtf(a[1] * per + c.eps) : 1.f;
    const float m1 = a[2] * rx * per, m0 = LAYER ? a[3] * per : 0.f;
    float ct = c.beta;
    if (c.gate_mode == MOE_GATE_TOKEN) ct *= load_w1(c.gate, c.w_f32, t);
    // D and n of the 8 values from j
    const auto point = [&](int j, float (&D)[kNV], float (&n)[kNV], float (&n2)[kNV], float (&dd)[kNV]) {
      const Vec<TR, kNV> xv = c.dh ? load_vec<TR, kNV>(x, j, N) : Vec<TR, kNV>{};
      const Vec<TZ, kNV> dv = c.dh ? load_vec<TZ, kNV>(dh, j, N) : Vec<TZ, kNV>{};
      const Vec<TZ, kNV> zv = c.z ? load_vec<TZ, kNV>(z, j, N) : Vec<TZ, kNV>{};
      const Vec<TR, kNV> rv = c.dr_out ? load_vec<TR, kNV>(dr, j, N) : Vec<TR, kNV>{};
      float w[kNV];
      load_w(c.w_pre, c.w_f32, j, N, w, 1.f);
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        n2[i] = (to_f32(xv.v[i]) - mx) * rx;
        dd[i] = to_f32(dv.v[i]);
        D[i] = to_f32(rv.v[i]) + (c.dh ? rx * (dd[i] * w[i] - n2[i] * m1 - m0) : 0.f);
        n[i] = (to_f32(zv.v[i]) - mz) * rz;
      }
    };
    float b[3] = {0.f, 0.f, 0.f};
    for (int j = threadIdx.x * kNV; j < N; j += step) {
      float D[kNV], n[kNV], n2[kNV], dd[kNV], wp[kNV], bp[kNV], g[kNV];
      point(j, D, n, n2, dd);
      load_w(c.w_post, c.w_f32, j, N, wp, 1.f);
      load_w(c.gate_mode == MOE_GATE_TOKEN ? c.b_post : nullptr, c.w_f32, j, N, bp, 0.f);
      load_w(c.gate_mode == MOE_GATE_CHANNEL ? c.gate : nullptr, c.w_f32, j, N, g, 1.f);
      Vec<TR, kNV> o;
      float add[kNormSums][kNV];
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        from_f32(c.alpha * D[i], o.v[i]);
        add[0][i] = dd[i] * n2[i];
        add[1][i] = dd[i];
        add[2][i] = ct * D[i] * n[i];
        add[3][i] = ct * D[i];
        if (j + i >= N) continue;
        const float e = ct * D[i] * g[i] * wp[i];
        b[0] = fmaf(e, n[i], b[0]);
        b[1] += e;
        b[2] = fmaf(D[i], fmaf(n[i], wp[i], bp[i]), b[2]);
      }
      if (c.dr != nullptr) store_vec<TR, kNV>((TR*)c.dr + at, j, N, o);
#pragma unroll
      for (int q = 0; q < kNormSums; ++q) {
        if (!(c.use >> q & 1)) continue;
        float* p = row + (int64_t)q * N;
        Vec<float, kNV> v = first ? Vec<float, kNV>{} : load_vec<float, kNV>(p, j, N);
#pragma unroll
        for (int i = 0; i < kNV; ++i) v.v[i] += add[q][i];
        store_vec<float, kNV>(p, j, N, v);
      }
    }
    if (c.z == nullptr) continue;
    row_sums<W, 3>(b, s, wr, slot);
    if (c.gate_mode == MOE_GATE_TOKEN && c.dgate != nullptr && threadIdx.x == 0) {
      if (c.dw_f32) ((float*)c.dgate)[t] = c.beta * b[2];
      else ((bf16_t*)c.dgate)[t] = f32_to_bf16(c.beta * b[2]);
    }
    if (c.dz == nullptr) continue;
    const float k1 = c.post ? b[0] * per : 0.f, k0 = LAYER && c.post ? b[1] * per : 0.f;
    for (int j = threadIdx.x * kNV; j < N; j += step) {
      float D[kNV], n[kNV], n2[kNV], dd[kNV], wp[kNV], g[kNV];
      point(j, D, n, n2, dd);
      load_w(c.w_post, c.w_f32, j, N, wp, 1.f);
      load_w(c.gate_mode == MOE_GATE_CHANNEL ? c.gate : nullptr, c.w_f32, j, N, g, 1.f);
      Vec<TZ, kNV> o;
#pragma unroll
      for (int i = 0; i < kNV; ++i) from_f32(rz * (ct * D[i] * g[i] * wp[i] - n[i] * k1 - k0), o.v[i]);
      store_vec<TZ, kNV>((TZ*)c.dz + at, j, N, o);
    }
  }
}

// The column sums of `rows` rows of partial sums: a block takes 64 columns, wave w
// rows w, w + 16, ...; the waves' sums are added in order.
__global__ __launch_bounds__(1024) void norm_finish_kernel(NormBwdCall c, int rows) {
  __shared__ float s[kNormSums][16][kWave];
  const int w = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int j = blockIdx.x * kWave + lane, N = c.N;
  float a[kNormSums] = {0.f, 0.f, 0.f, 0.f};
  if (j < N) {
#pragma unroll
    for (int q = 0; q < kNormSums; ++q)
      if (c.use >> q & 1) {
        const float* p = c.sums + (int64_t)q * N + j;
#pragma unroll 8
        for (int r = w; r < rows; r += 16) a[q] += p[(int64_t)r * kNormSums * N];
      }
  }
#pragma unroll
  for (int q = 0; q < kNormSums; ++q) s[q][w][lane] = a[q];
  __syncthreads();
  if (w != 0 || j >= N) return;
#pragma unroll
  for (int q = 0; q < kNormSums; ++q) {
    a[q] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a[q] += s[q][i][lane];
  }
  const auto put = [&](void* out, float v) {
    if (out == nullptr) return;
    if (c.dw_f32) ((float*)out)[j] = v;
    else ((bf16_t*)out)[j] = f32_to_bf16(v);
  };
  put(c.dw_pre, a[0]);
  put(c.db_pre, a[1]);
  const float g = c.gate_mode == MOE_GATE_CHANNEL ? load_w1(c.gate, c.w_f32, j) : 1.f;
  put(c.dw_post, g * a[2]);
  put(c.db_post, g * a[3]);
  if (c.gate_mode == MOE_GATE_CHANNEL) {
    const float w1 = c.w_post ? load_w1(c.w_post, c.w_f32, j) : 1.f;
    const float b1 = c.b_post ? load_w1(c.b_post, c.w_f32, j) : 0.f;
    put(c.dgate, fmaf(w1, a[2], b1 * a[3]));
  }
}

// Waves per row and accesses per lane: one wave where it holds the row in 8
// accesses and there are rows enough to occupy the GPU, else more waves.
struct NormPlan {
  int W, C;
};
NormPlan norm_plan(int64_t T, int N) {
  const int need = (N + kNV * kWave - 1) / (kNV * kWave);  // accesses of one wave
  const auto pow2 = [](int v) { int p = 1; while (p < v) p *= 2; return p; };
  if (need <= 8 && (T >= 2048 || need == 1)) return {1, pow2(need)};
  if (need <= 32 && T >= 512) return {4, pow2((need + 3) / 4)};
  if (need <= 4) return {4, 1};
  return {16, pow2((need + 15) / 16)};
}

template <typename TZ, typename TR, int W, int C>
void go_norm(const NormCall& c, hipStream_t s) {
  constexpr int rows = W > 4 ? 1 : 4 / W;
  hipLaunchKernelGGL((norm_kernel<TZ, TR, W, C>), dim3((unsigned)cdiv64(c.T, rows)), dim3(W > 4 ? W * kWave : 256), 0,
                     s, c);
}

template <typename TZ, typename TR>
void pick_norm(const NormCall& c, hipStream_t s) {
  const NormPlan p = norm_plan(c.T, c.N);
#define MOE_NORM(w, n) if (p.W == w && p.C == n) return go_norm<TZ, TR, w, n>(c, s)
  MOE_NORM(1, 1); MOE_NORM(1, 2); MOE_NORM(1, 4); MOE_NORM(1, 8);
  MOE_NORM(4, 1); MOE_NORM(4, 2); MOE_NORM(4, 4); MOE_NORM(4, 8);
  MOE_NORM(16, 1); MOE_NORM(16, 2); MOE_NORM(16, 4); MOE_NORM(16, 8);
#undef MOE_NORM
}

// Backward: W waves to a row, C accesses to a lane (C = 0: the wide kernel), blocks,
// and rows of partial sums.
struct NormBwdPlan {
  int W, C, blocks, parts;
};
NormBwdPlan norm_bwd_plan(int64_t T, int N) {
  const int need = (N + kNV * kWave - 1) / (kNV * kWave);
  NormBwdPlan p;
  p.W = 1;
  while (p.W < need && p.W < 16) p.W *= 2;
  p.C = need <= 16 ? 1 : need <= 32 ? 2 : 0;
  const int rows = p.W > 4 ? 1 : 4 / p.W;
  const int64_t most = 4096 / (p.W * rows);
  const int64_t all = cdiv64(T, rows);
  p.blocks = (int)(all < most ? all : most);
  p.parts = p.blocks * rows;
  return p;
}

template <typename TZ, typename TR, bool LAYER>
void pick_norm_bwd(const NormBwdCall& c, const NormBwdPlan& p, hipStream_t s) {
#define MOE_NORM(w, n)                                                                                       \
  if (p.W == w && p.C == n) {                                                                                \
    hipLaunchKernelGGL((norm_bwd_kernel<TZ, TR, LAYER, w, n>), dim3(p.blocks), dim3(w > 4 ? w * kWave : 256), \
                       0, s, c);                                                                             \
    return;                                                                                                  \
  }
  MOE_NORM(1, 1) MOE_NORM(2, 1) MOE_NORM(4, 1) MOE_NORM(8, 1) MOE_NORM(16, 1) MOE_NORM(16, 2)
#undef MOE_NORM
  hipLaunchKernelGGL((norm_bwd_wide_kernel<TZ, TR, LAYER>), dim3(p.blocks), dim3(1024), 0, s, c);
}

template <typename TZ, typename TR>
void pick_norm_bwd_kind(const NormBwdCall& c, const NormBwdPlan& p, hipStream_t s) {
  if (c.kind == MOE_NORM_LAYER) pick_norm_bwd<TZ, TR, true>(c, p, s);
  else pick_norm_bwd<TZ, TR, false>(c, p, s);
}

}  // namespace

size_t norm_bwd_ws_bytes(int T, int N) {
  if (T == 0) return 0;
  return (size_t)norm_bwd_plan(T, N).parts * kNormSums * N * 4;
}

moe_status launch_norm_bwd(NormBwdCall c, moe_dtype dt, moe_dtype r_dt, hipStream_t s) {
  const bool channel = c.gate_mode == MOE_GATE_CHANNEL && c.dgate != nullptr;
  c.use = (c.dw_pre ? 1 : 0) | (c.db_pre ? 2 : 0) | (c.dw_post || channel ? 4 : 0) |
          (c.db_post || (channel && c.b_post) ? 8 : 0);
  if (!c.use) c.sums = nullptr;
  int parts = 0;
  if (c.T > 0) {
    const NormBwdPlan p = norm_bwd_plan(c.T, c.N);
    parts = p.parts;
    if (dt == MOE_F32) pick_norm_bwd_kind<float, float>(c, p, s);
    else if (r_dt == MOE_F32) pick_norm_bwd_kind<bf16_t, float>(c, p, s);
    else pick_norm_bwd_kind<bf16_t, bf16_t>(c, p, s);
  }
  if (c.use) hipLaunchKernelGGL(norm_finish_kernel, dim3(cdiv(c.N, kWave)), dim3(1024), 0, s, c, parts);
  return launch_status();
}

moe_status launch_norm(const NormCall& c, moe_dtype dt, moe_dtype r_dt, hipStream_t s) {
  if (c.T == 0) return MOE_OK;
  if (dt == MOE_F32) pick_norm<float, float>(c, s);
  else if (r_dt == MOE_F32) pick_norm<bf16_t, float>(c, s);
  else pick_norm<bf16_t, bf16_t>(c, s);
  return launch_status();
}

}  // namespace moe
