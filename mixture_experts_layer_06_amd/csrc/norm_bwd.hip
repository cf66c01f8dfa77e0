// norm_bwd.hip — the gradients of the norms around a block (norm.hip): their formulas
// stand there.
//
// One pass: a block holds a row and its columns' sums in registers and walks rows a grid
// apart, so that the sums over tokens leave it once. 8192 x 4096, bf16 with a binary32
// residual, RMS norms, gate per channel: 110 us, 5.7 TB/s of HBM traffic, and 8 us to add
// up the blocks' sums (34 MB). Layer norms have two sums more to a column: over 2048
// columns they and what 8 or 16 waves hold of a row exceed the registers, and some of
// them live in scratch memory where that measured faster than the other forms below.
#include "norm.h"

namespace moe {
namespace {

// Sums over a block's rows go to its four rows of the workspace (of dh n', dh, S1's
// and S0's terms), N apart; the finishing launch adds the blocks' in order.
constexpr int kNormSums = 4;

// Two blocks of 8 waves share a CU; layer norms of rows off 16 bytes take the registers of
// both (2000 x 4095, bf16: 67 us against 84; aligned rows 55 against 52).
template <typename TZ, typename TR, bool LAYER, int W, int C, int MODE>
__global__ __launch_bounds__(W > 4 ? W * kWave : 256, W != 8 ? 0 : LAYER && MODE != kWhole ? 2 : 4)
void norm_bwd_kernel(NormBwdCall c) {
  constexpr int kRows = W > 4 ? 1 : 4 / W;
  __shared__ __attribute__((aligned(16))) float s[kRows][2][W][4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wr = wave % W, sub = wave / W;
  const int N = c.N;
  const auto col = [&](int q) { return ((q * W + wr) * kWave + (int)threadIdx.x % kWave) * kNV; };
  const auto on = [&](int q, int i) { return MODE == kWhole ? col(q) < N : col(q) + i < N; };
  const float per = 1.f / (float)N;
  float d1[C][kNV], d0[C][kNV], s1[C][kNV], s0[C][kNV];
#pragma unroll
  for (int q = 0; q < C; ++q)
#pragma unroll
    for (int i = 0; i < kNV; ++i) d1[q][i] = d0[q][i] = s1[q][i] = s0[q][i] = 0.f;
  int slot = 0;
  // What was loaded stays in its type and is widened again at each use: the registers
  // it would take as binary32 are waves that hide the memory's latency. Registers whose
  // row is used up take the block's next row at once (8192 x 4096 bf16: 103 -> 93 us,
  // 8192 x 1501: 84 -> 60), but not where the sums of a layer norm leave too few for
  // two blocks of a CU (151 -> 171).
  constexpr bool kAhead = C == 1 && (!LAYER || W <= 4);
  RowVec<TR, kNV, MODE, MODE == kWhole> x[C], rv[C];
  RowVec<TZ, kNV, MODE, MODE == kWhole> dd[C], z[C];
  const auto row_of = [&](int64_t tb) { return (tb + sub < c.T ? tb + sub : 0) * N; };  // row 0 for rows past the last
  const auto load_r = [&](int64_t at) {
#pragma unroll
    for (int q = 0; q < C; ++q) {
      if (c.dh != nullptr) {
        x[q].load((const TR*)c.r_out + at, col(q), N);
        dd[q].load((const TZ*)c.dh + at, col(q), N);
      }
      if (c.dr_out != nullptr) rv[q].load((const TR*)c.dr_out + at, col(q), N);
    }
  };
  const auto load_z = [&](int64_t at) {
    if (c.z != nullptr)
#pragma unroll
      for (int q = 0; q < C; ++q) z[q].load((const TZ*)c.z + at, col(q), N);
  };
#pragma unroll
  for (int q = 0; q < C; ++q) x[q].zero(), rv[q].zero(), dd[q].zero(), z[q].zero();
  const int64_t step = (int64_t)gridDim.x * kRows;
  const bool token = c.gate_mode == MOE_GATE_TOKEN;
  // this lane's columns' factors, w_pre and w_post times the channels' gate: once for
  // all of its rows where the registers are there (8192 x 4096: 135 -> 123 us)
  constexpr bool kKeep = C == 1;
  float wq[C][kNV], gw[C][kNV];
  const auto load_wq = [&](int q) { load_w<MODE>(c.w_pre, c.w_f32, col(q), N, wq[q], 1.f); };
  const auto load_gw = [&](int q) {
    float g[kNV];
    load_w<MODE>(c.w_post, c.w_f32, col(q), N, gw[q], 1.f);
    load_w<MODE>(c.gate_mode == MOE_GATE_CHANNEL ? c.gate : nullptr, c.w_f32, col(q), N, g, 1.f);
#pragma unroll
    for (int i = 0; i < kNV; ++i) gw[q][i] *= g[i];
  };
  if (kKeep) {
    load_wq(0);
    load_gw(0);
  }
  load_r(row_of((int64_t)blockIdx.x * kRows));
  load_z(row_of((int64_t)blockIdx.x * kRows));
  // the rows of a block are walked by all of its waves together: the barriers match
  for (int64_t tb = (int64_t)blockIdx.x * kRows; tb < c.T; tb += step) {
    const int64_t t = tb + sub;
    const bool in = t < c.T;
    const int64_t at = row_of(tb);
    if (!kAhead && tb != (int64_t)blockIdx.x * kRows) {
      load_r(at);
      load_z(at);
    }
#pragma unroll
    for (int q = 0; q < C; ++q) {
      x[q].fix(col(q), N), dd[q].fix(col(q), N), z[q].fix(col(q), N), rv[q].fix(col(q), N);
    }
    float mx = 0.f, mz = 0.f;
    if (LAYER) {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int q = 0; q < C; ++q)
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          m[0] += x[q].at(i);
          m[1] += z[q].at(i);
        }
      row_sums<W, 2>(m, s[sub], wr, slot);
      mx = m[0] * per;
      mz = c.post ? m[1] * per : 0.f;
    }
    // squares of the two rows, and what pre's gradient needs of e = dh w
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < C; ++q) {
      if (!kKeep) load_wq(q);
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const float xc = LAYER && !on(q, i) ? 0.f : x[q].at(i) - mx;
        const float zc = LAYER && !on(q, i) ? 0.f : z[q].at(i) - mz;
        const float e = dd[q].at(i) * wq[q][i];
        a[0] = fmaf(xc, xc, a[0]);
        a[1] = fmaf(zc, zc, a[1]);
        a[2] = fmaf(e, xc, a[2]);
        if (LAYER) a[3] += e;
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
    float du[C][kNV];
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int j = col(q);
      float o[kNV];
      if (c.dh != nullptr) {
        if (!kKeep) load_wq(q);
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          const float n2 = (x[q].at(i) - mx) * rx, d = dd[q].at(i);
          du[q][i] = rv[q].at(i) + rx * (d * wq[q][i] - n2 * m1 - m0);
          if (in) {
            d1[q][i] = fmaf(d, n2, d1[q][i]);
            if (LAYER) d0[q][i] += d;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kNV; ++i) du[q][i] = rv[q].at(i);
      }
#pragma unroll
      for (int i = 0; i < kNV; ++i) o[i] = c.alpha * du[q][i];
      if (c.dr != nullptr && in) {
        RowVec<TR, kNV, MODE, MODE == kWhole> out;
        out.put(o);
        out.store((TR*)c.dr + at, j, N);
      }
      if (c.z == nullptr) continue;
      if (!kKeep) load_gw(q);
      if (token) {
#pragma unroll
        for (int i = 0; i < kNV; ++i)
          if (on(q, i)) b[2] = fmaf(du[q][i], (z[q].at(i) - mz) * rz * gw[q][i], b[2]);
        if (LAYER && c.b_post != nullptr) {
          float p[kNV];
          load_w<MODE>(c.b_post, c.w_f32, j, N, p, 0.f);
#pragma unroll
          for (int i = 0; i < kNV; ++i)
            if (on(q, i)) b[2] = fmaf(du[q][i], p[i], b[2]);
        }
      }
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const float n = (z[q].at(i) - mz) * rz, cd = ct * du[q][i];
        if (in) {
          s1[q][i] = fmaf(cd, n, s1[q][i]);
          if (LAYER) s0[q][i] += cd;
        }
        du[q][i] = cd * gw[q][i];  // w_post's factor too
        if (on(q, i)) {
          b[0] = fmaf(du[q][i], n, b[0]);
          if (LAYER) b[1] += du[q][i];
        }
      }
    }
    if (kAhead && tb + step < c.T) load_r(row_of(tb + step));
    if (c.z == nullptr) continue;
    row_sums<W, 3>(b, s[sub], wr, slot);
    if (c.gate_mode == MOE_GATE_TOKEN && c.dgate != nullptr && in && wr == 0 && threadIdx.x % kWave == 0) {
      const float dg = c.beta * b[2];
      if (c.dw_f32) ((float*)c.dgate)[t] = dg;
      else ((bf16_t*)c.dgate)[t] = f32_to_bf16(dg);
    }
    const float k1 = c.post ? b[0] * per : 0.f, k0 = LAYER && c.post ? b[1] * per : 0.f;
    if (c.dz != nullptr && in)
#pragma unroll
      for (int q = 0; q < C; ++q) {
        float o[kNV];
#pragma unroll
        for (int i = 0; i < kNV; ++i) o[i] = rz * (du[q][i] - (z[q].at(i) - mz) * rz * k1 - k0);
        RowVec<TZ, kNV, MODE, MODE == kWhole> out;
        out.put(o);
        out.store((TZ*)c.dz + at, col(q), N);
      }
    if (kAhead && tb + step < c.T) load_z(row_of(tb + step));
  }
  if (c.sums == nullptr) return;
  // the block's rows meet in LDS, so that it leaves one row of sums
  float* row = c.sums + (int64_t)blockIdx.x * kNormSums * N;
  const auto put = [&](int which, float (&v)[C][kNV]) {
    if (!(c.use >> which & 1)) return;
    if constexpr (kRows > 1) {
      __shared__ float all[kRows - 1][kNV][W * kWave];
      const int lane = wr * kWave + threadIdx.x % kWave;
      __syncthreads();
      if (sub > 0)
#pragma unroll
        for (int i = 0; i < kNV; ++i) all[sub - 1][i][lane] = v[0][i];
      __syncthreads();
      if (sub > 0) return;
#pragma unroll
      for (int r = 0; r < kRows - 1; ++r)
#pragma unroll
        for (int i = 0; i < kNV; ++i) v[0][i] += all[r][i][lane];
    }
#pragma unroll
    for (int q = 0; q < C; ++q) {
      RowVec<float, kNV, MODE> o;
      o.put(v[q]);
      o.store(row + (int64_t)which * N, col(q), N);
    }
  };
  put(0, d1);
  if (LAYER) put(1, d0);
  put(2, s1);
  if (LAYER) put(3, s0);
}

// Rows wider than the registers hold: a block of 16 waves per row, read again from
// memory (the caches) at each of its steps; the block's sums live in its rows of the
// workspace, each column touched by one lane only.
template <typename TZ, typename TR, bool LAYER, int MODE>
__global__ __launch_bounds__(1024) void norm_bwd_wide_kernel(NormBwdCall c) {
  constexpr int W = 16;
  typedef RowVec<TZ, kNV, MODE> Z;
  typedef RowVec<TR, kNV, MODE> V;
  __shared__ __attribute__((aligned(16))) float s[2][W][4];
  const int wr = threadIdx.x / kWave;
  const int N = c.N, step = 1024 * kNV;
  const float per = 1.f / (float)N;
  float* row = c.sums ? c.sums + (int64_t)blockIdx.x * kNormSums * N : nullptr;
  int slot = 0;
  bool first = true;
  // 8 values of a row, zeros where there is none
  const auto read = [&](bool there, const auto* row, int j, float (&o)[kNV], auto v) {
    if (there) v.load(row, j, N);
    else v.zero();
    v.get(o, j, N);
  };
  for (int64_t t = blockIdx.x; t < c.T; t += gridDim.x, first = false) {
    const int64_t at = t * N;
    const TZ* dh = (const TZ*)c.dh + at;
    const TZ* z = (const TZ*)c.z + at;
    const TR* x = (const TR*)c.r_out + at;
    const TR* dr = (const TR*)c.dr_out + at;
    float m[2] = {0.f, 0.f};
    if (LAYER) {
      for (int j = threadIdx.x * kNV; j < N; j += step) {
        float xv[kNV], zv[kNV];
        read(c.dh != nullptr, x, j, xv, V{});
        read(c.post, z, j, zv, Z{});
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          m[0] += xv[i];
          m[1] += zv[i];
        }
      }
      row_sums<W, 2>(m, s, wr, slot);
    }
    const float mx = m[0] * per, mz = m[1] * per;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = threadIdx.x * kNV; j < N; j += step) {
      float xv[kNV], dv[kNV], zv[kNV], w[kNV];
      read(c.dh != nullptr, x, j, xv, V{});
      read(c.dh != nullptr, dh, j, dv, Z{});
      read(c.post, z, j, zv, Z{});
      load_w<MODE>(c.w_pre, c.w_f32, j, N, w, 1.f);
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        if (j + i >= N) continue;
        const float xc = xv[i] - mx, zc = zv[i] - mz, e = dv[i] * w[i];
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
      float w[kNV];
      read(c.dh != nullptr, x, j, n2, V{});
      read(c.dh != nullptr, dh, j, dd, Z{});
      read(c.z != nullptr, z, j, n, Z{});
      read(c.dr_out != nullptr, dr, j, D, V{});
      load_w<MODE>(c.w_pre, c.w_f32, j, N, w, 1.f);
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        n2[i] = (n2[i] - mx) * rx;
        if (c.dh != nullptr) D[i] += rx * (dd[i] * w[i] - n2[i] * m1 - m0);
        n[i] = (n[i] - mz) * rz;
      }
    };
    float b[3] = {0.f, 0.f, 0.f};
    for (int j = threadIdx.x * kNV; j < N; j += step) {
      float D[kNV], n[kNV], n2[kNV], dd[kNV], wp[kNV], bp[kNV], g[kNV];
      point(j, D, n, n2, dd);
      load_w<MODE>(c.w_post, c.w_f32, j, N, wp, 1.f);
      load_w<MODE>(c.gate_mode == MOE_GATE_TOKEN ? c.b_post : nullptr, c.w_f32, j, N, bp, 0.f);
      load_w<MODE>(c.gate_mode == MOE_GATE_CHANNEL ? c.gate : nullptr, c.w_f32, j, N, g, 1.f);
      float o[kNV], add[kNormSums][kNV];
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        o[i] = c.alpha * D[i];
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
      if (c.dr != nullptr) {
        V out;
        out.put(o);
        out.store((TR*)c.dr + at, j, N);
      }
#pragma unroll
      for (int q = 0; q < kNormSums; ++q) {
        if (!(c.use >> q & 1)) continue;
        float* p = row + (int64_t)q * N;
        float had[kNV];
        RowVec<float, kNV, MODE> v;
        read(!first, p, j, had, v);
#pragma unroll
        for (int i = 0; i < kNV; ++i) had[i] += add[q][i];
        v.put(had);
        v.store(p, j, N);
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
      load_w<MODE>(c.w_post, c.w_f32, j, N, wp, 1.f);
      load_w<MODE>(c.gate_mode == MOE_GATE_CHANNEL ? c.gate : nullptr, c.w_f32, j, N, g, 1.f);
      float o[kNV];
#pragma unroll
      for (int i = 0; i < kNV; ++i) o[i] = rz * (ct * D[i] * g[i] * wp[i] - n[i] * k1 - k0);
      Z out;
      out.put(o);
      out.store((TZ*)c.dz + at, j, N);
    }
  }
}

// The column sums of `rows` rows of partial sums: a block takes 16 columns, 64 runs
// of rows to each (run g: rows g, g + 64, ...), so that many blocks have short ways;
// the runs' sums are added in a fixed order.
__global__ __launch_bounds__(1024) void norm_finish_kernel(NormBwdCall c, int rows) {
  __shared__ float s[kNormSums][16][16];
  const int w = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int j = blockIdx.x * 16 + lane % 16, N = c.N;
  float a[kNormSums] = {0.f, 0.f, 0.f, 0.f};
  if (j < N) {
#pragma unroll
    for (int q = 0; q < kNormSums; ++q)
      if (c.use >> q & 1) {
        const float* p = c.sums + (int64_t)q * N + j;
#pragma unroll 8
        for (int r = w * 4 + lane / 16; r < rows; r += 64) a[q] += p[(int64_t)r * kNormSums * N];
      }
  }
#pragma unroll
  for (int q = 0; q < kNormSums; ++q) {
    a[q] += __shfl_xor(a[q], 16, kWave);
    a[q] += __shfl_xor(a[q], 32, kWave);
    if (lane < 16) s[q][w][lane] = a[q];
  }
  __syncthreads();
  if (threadIdx.x >= 16 || j >= N) return;
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

// W waves to a row, C accesses to a lane (C = 0: the wide kernel; of C = 2 layer norms
// only some, below), and blocks, each of
// which walks its share of the rows and leaves a row of sums: enough to occupy the
// GPU (16 waves per CU), but at least four rows to a block where there are 256 blocks
// (1024 x 4096: 24 us, at two rows 26; 2048 x 2048: 24 and 26).
struct NormBwdPlan {
  int W, C, blocks;
};
NormBwdPlan norm_bwd_plan(int64_t T, int N) {
  const int need = (N + kNV * kWave - 1) / (kNV * kWave);
  NormBwdPlan p;
  p.W = 1;
  while (p.W < need && p.W < 16) p.W *= 2;
  p.C = need <= 16 ? 1 : need <= 32 ? 2 : 0;
  const int rows = p.W > 4 ? 1 : 4 / p.W;
  const int64_t most = 4096 / (p.W * rows), all = cdiv64(T, rows);
  const int64_t few = all / 4 > 256 ? all / 4 : 256;
  p.blocks = (int)(all < few ? all : few < most ? few : most);
  return p;
}

template <typename TZ, typename TR, bool LAYER, int MODE>
void pick_norm_bwd(const NormBwdCall& c, const NormBwdPlan& p, hipStream_t s) {
#define MOE_NORM(w, n)                                                                                    \
  if (p.W == w && p.C == n) {                                                                             \
    if constexpr (MODE != kNarrow || w == 1)                                                              \
      hipLaunchKernelGGL((norm_bwd_kernel<TZ, TR, LAYER, w, n, MODE>), dim3(p.blocks),                    \
                         dim3(w > 4 ? w * kWave : 256), 0, s, c);                                         \
    return;                                                                                               \
  }
  MOE_NORM(1, 1) MOE_NORM(2, 1) MOE_NORM(4, 1) MOE_NORM(8, 1) MOE_NORM(16, 1)
  // Two accesses to a lane spill: RMS norms least (1500 x 12288, bf16: 96 us, the wide
  // kernel 137; binary32 197 and 200), layer norms so that the wide kernel is faster (8200
  // wide, bf16: 140 us against 190, binary32 189 against 310; 12288 wide, bf16: 195 against
  // 208), but for the longest bf16 rows on 16 bytes (16384 wide: 259 against 234).
  if constexpr (!LAYER || (MODE == kWhole && sizeof(TZ) == 2)) {
    if (!LAYER || c.N > 14336) {
      MOE_NORM(16, 2)
    }
  }
#undef MOE_NORM
  if constexpr (MODE != kNarrow)
    hipLaunchKernelGGL((norm_bwd_wide_kernel<TZ, TR, LAYER, MODE>), dim3(p.blocks), dim3(1024), 0, s, c);
}

template <typename TZ, typename TR>
void pick_norm_bwd_kind(const NormBwdCall& c, const NormBwdPlan& p, hipStream_t s) {
  with_mode(row_mode(c.N, kNV), [&](auto mode) {
    if (c.kind == MOE_NORM_LAYER) pick_norm_bwd<TZ, TR, true, mode()>(c, p, s);
    else pick_norm_bwd<TZ, TR, false, mode()>(c, p, s);
  });
}

}  // namespace

size_t norm_bwd_ws_bytes(int T, int N) {
  if (T == 0) return 0;
  return (size_t)norm_bwd_plan(T, N).blocks * kNormSums * N * 4;
}

moe_status launch_norm_bwd(NormBwdCall c, moe_dtype dt, moe_dtype r_dt, hipStream_t s) {
  const bool channel = c.gate_mode == MOE_GATE_CHANNEL && c.dgate != nullptr;
  c.use = (c.dw_pre ? 1 : 0) | (c.db_pre ? 2 : 0) | (c.dw_post || channel ? 4 : 0) |
          (c.db_post || (channel && c.b_post) ? 8 : 0);
  if (!c.use) c.sums = nullptr;
  const NormBwdPlan p = norm_bwd_plan(c.T, c.N);
  if (c.T > 0) {
    if (dt == MOE_F32) pick_norm_bwd_kind<float, float>(c, p, s);
    else if (r_dt == MOE_F32) pick_norm_bwd_kind<bf16_t, float>(c, p, s);
    else pick_norm_bwd_kind<bf16_t, bf16_t>(c, p, s);
  }
  if (c.use) hipLaunchKernelGGL(norm_finish_kernel, dim3(cdiv(c.N, 16)), dim3(1024), 0, s, c, p.blocks);
  return launch_status();
}

}  // namespace moe
