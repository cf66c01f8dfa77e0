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
// One card, bf16, us: 8192 rows 7168 -> 2048, rank 64, 8 adapters 34 + 8 + 27 (down,
// pack, up; 5.1 TB/s of HBM traffic in down, whose adapters each XCD reads for itself);
// back through 4096 -> 4096, rank 16, 4 adapters 21 + 5 + 35 + 37 + 5 (3.5 to 4.0 TB/s
// in down, up and grad); 64 rows of 32 adapters 4096 -> 4096, rank 16 5 + 7, where a
// block's chain of loads is the time.
//
// u and du are binary32. A bf16 MFMA takes them as two bf16 terms, u = hi + lo with
// lo = bf16(u - hi): 16 bits of u, so that a bf16 result carries one rounding, its
// own, where u rounded once to bf16 would add another of its size. The products
// double, which the memory's time hides. Weight gradients that are stored in binary32
// take three terms, all 24 bits. fp32 tensors use the fp32 MFMA.
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

template <typename T, int MODE, bool STREAM>
__device__ __forceinline__ typename Frag8<T>::Type frag_of(const RowVec<T, 8, MODE, STREAM>& v) {
  return __builtin_bit_cast(typename Frag8<T>::Type, v.w);
}

// The upper bf16 terms of x and y as one word; x and y become what these leave. A value
// between bf16's and binary32's largest takes bf16's largest, where rounding would give
// an infinity and leave the other one; what is infinite or no number leaves nothing.
__device__ __forceinline__ uint32_t upper_terms(float& x, float& y) {
  constexpr float kLast = 0x1.fep127f, kMax = 0x1.fffffep127f;
  const bool fx = fabsf(x) <= kMax, fy = fabsf(y) <= kMax;
  const uint32_t w = pack_bf16x2(fx ? __builtin_amdgcn_fmed3f(x, -kLast, kLast) : x,
                                 fy ? __builtin_amdgcn_fmed3f(y, -kLast, kLast) : y);
  x = fx ? x - __uint_as_float(w << 16) : 0.f;
  y = fy ? y - __uint_as_float(w & 0xffff0000u) : 0.f;
  return w;
}

// Ranks of a row of u in the workspace.
__host__ __device__ constexpr int padded(int R) { return (R + 7) & ~7; }

// The tensors' row of grouped row r, or -1. Always one load, so that several can be in
// flight.
__device__ __forceinline__ int row_entry(const LoraCall& c, int r) {
  return c.rows != nullptr ? c.rows[r] : c.offsets[0];
}
__device__ __forceinline__ int row_of(const LoraCall& c, int r, int entry) {
  const int t = c.rows != nullptr ? entry : r;
  return t >= 0 && t < c.T ? t : -1;
}

// Which of the tensors' rows the list names, for calls that fill the others, without
// clearing anything first: entry r leaves its number at its row's place, and a row is
// listed if the entry that its place names names it back. What the place of another row
// holds is any number at all.
// With all rows listed the check is not seen (8192 rows 7168 -> 2048, rank 64: 70 us with
// and without); base copied first would take longer there, and as long where few are
// (512 of 8192 x 4096: 46 us, copied first 39; 8 of 64: 9.1 and 11.2).
constexpr int kMarkRows = 1024;  // entries of a block that marks
constexpr int kFillRows = 16;    // rows of a block that fills
__device__ __forceinline__ void mark_rows(const LoraCall& c, int block) {
#pragma unroll
  for (int i = 0; i < kMarkRows / 256; ++i) {
    const int r = block * kMarkRows + i * 256 + (int)threadIdx.x;
    const int t = r < c.M ? c.rows[r] : -1;
    if (t >= 0 && t < c.T) c.listed[t] = r;
  }
}
__device__ __forceinline__ bool is_listed(const LoraCall& c, int t) {
  const int r = c.listed[t];
  return r >= 0 && r < c.M && c.rows[r] == t;
}

// 8 ranks from j on of N rows of R, zeros past them, all loads before their first use.
// R8: R is a multiple of 8; otherwise halves (R = 4, 12, ..) or single ranks, whose
// branch makes the compiler wait for them at once.
template <typename T, bool R8>
struct Ranks {
  static constexpr int kWords = 2 * (int)sizeof(T);
  RowVec<T, 8, R8 ? kWhole : kNarrow> x;
  template <int N, typename A>
  static __device__ __forceinline__ void load(Ranks (&v)[N], int R, A at) {  // at(i, row, j): where v[i] lies
    if (R8 || R % 4 != 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const T* row;
        int j;
        at(i, row, j);
        v[i].x.load(row, j, R);
      }
    } else {
      RowVec<T, 4, kWhole> half[N][2];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const T* row;
        int j;
        at(i, row, j);
        half[i][0].load(row, j, R);
        half[i][1].load(row, j + 4, R);
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < kWords; ++k) v[i].x.w[k] = half[i][k / (kWords / 2)].w[k % (kWords / 2)];
    }
  }
  __device__ __forceinline__ void fix(int j, int R) { x.fix(j, R); }  // ranks past R become zeros
};

// Block p runs on XCD p % 8: logical position L of `total`, each XCD taking a run of
// them, so that the column tiles of a row meet in one L2 and every L2 sees all of
// the row's columns (with neighbouring tiles on different XCDs each L2 saw the same
// few columns of every row, and a quarter of its channels did the work). False: none.
// The grid has a multiple of 8 blocks, at least `total`.
__device__ __forceinline__ bool xcd_run(int p, int total, int& L) {
  const int per = (total + 7) / 8;
  L = (p & 7) * per + (p >> 3);
  return (p >> 3) < per && L < total;
}

// ------------------------------------------------------------------ rows times (K,R)

// A tile: RW waves of XF fragments of 16 rows each, all F fragments of ranks; the
// other waves of the block (KW = 4 / RW teams) take other slices of k.
template <typename T, int F, int RW, int XF, bool WK>
struct DownCfg {
  static constexpr int kBM = RW * XF * 16, kKW = 4 / RW;
  // k of a slice: as deep as the loads in flight need and the ring's LDS allows
  static constexpr int kTK = RW == 1 ? (F * sizeof(T) >= 8 ? 32 : 64) : F * sizeof(T) >= 16 ? 64 : 128;
  static constexpr int kR = F * 16;                 // ranks, padded
  static constexpr int kPitch = sizeof(T) == 2 ? kR * 2 : (kR + 4) * 4;  // bytes of a k row in LDS
  static constexpr int kTile = kTK * kPitch;
  static constexpr int kTeam = 256 / kKW;           // threads
  static constexpr int kRing = WK ? 0 : kKW * 2 * kTile, kAcc = kKW > 1 ? 4 * F * kWave * 16 : 0;
  static constexpr int kLds = kRing > kAcc ? kRing : kAcc > 0 ? kAcc : 16;
};

template <typename T, int F, int RW, int XF, bool WK, int MODE, bool R8>
__global__ __launch_bounds__(256) void down_kernel(LoraCall c, const T* __restrict__ x, const T* __restrict__ w, int K,
                                                   int split, int range, float* __restrict__ part,
                                                   float* __restrict__ exact) {
  typedef DownCfg<T, F, RW, XF, WK> C;
  typedef typename Frag8<T>::Type Frag;
  if ((int)blockIdx.y == split) {  // behind all tiles: for the launch after
    mark_rows(c, blockIdx.x);
    return;
  }
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
    const int m = (rw * XF + i) * 16 + ci, r = tile.row0 + min(m, tile.rows - 1);
    const int t = row_of(c, r, row_entry(c, r));
    there[i] = t >= 0 && m < tile.rows;
    xr[i] = x + (int64_t)(there[i] ? t : 0) * K;
  }
  constexpr int kQ = C::kTK / 32;
  typedef RowVec<T, 8, MODE> X;  // half cache lines: the next access takes the other half from the cache
  X xv[2][XF][kQ];  // two slices: the loads of one last longer than the products of the other
  const auto load_x = [&](X (&v)[XF][kQ], int k0) {
#pragma unroll
    for (int i = 0; i < XF; ++i)
#pragma unroll
      for (int s = 0; s < kQ; ++s) v[i][s].load(xr[i], k0 + 32 * s + 8 * q, k_hi);
  };
  // a slice of the matrix in registers on its way to LDS: 8 ranks of a k row each
  constexpr int kPieces = C::kTK * C::kR / 8, kWV = kPieces > C::kTeam ? kPieces / C::kTeam : 1;
  static_assert(kPieces % C::kTeam == 0 || kPieces < C::kTeam, "whole pieces");
  typedef Ranks<T, R8> V;
  constexpr bool kEarly = kWV * 2 * (int)sizeof(T) <= 16;  // a slice ahead while it fits the registers
  constexpr int kHeld = WK ? 1 : kEarly ? kWV : 2;
  V wv[kHeld];
  const auto piece_k = [&](int u) { return (tt + u * C::kTeam) / (C::kR / 8); };
  const auto piece_j = [&](int u) { return (tt + u * C::kTeam) % (C::kR / 8) * 8; };
  const auto load_w = [&](int k0, int u0) {
    V::load(wv, R, [&](int u, const T*& row, int& j) {
      row = we + (int64_t)min(k0 + piece_k(u0 + u), k_hi - 1) * R;
      j = piece_j(u0 + u);
    });
  };
  const auto put_held = [&](unsigned char* t, int k0, int u0) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int k = piece_k(u0 + u), j = piece_j(u0 + u);
      if (kPieces < C::kTeam && tt >= kPieces) return;
      wv[u].fix(j, R);
      const bool on = k0 + k < k_hi;
      uint4* p = reinterpret_cast<uint4*>(t + k * C::kPitch + j * (int)sizeof(T));
#pragma unroll
      for (int h = 0; h < (int)sizeof(T) / 2; ++h)
        p[h] = make_uint4(on ? wv[u].x.w[4 * h] : 0u, on ? wv[u].x.w[4 * h + 1] : 0u, on ? wv[u].x.w[4 * h + 2] : 0u,
                          on ? wv[u].x.w[4 * h + 3] : 0u);
    }
  };
  const auto put_w = [&](unsigned char* t, int k0) {
    if constexpr (kEarly) {
      put_held(t, k0, 0);
    } else {
#pragma unroll 1
      for (int u = 0; u < kWV; u += kHeld) {
        load_w(k0, u);
        put_held(t, k0, u);
      }
    }
  };
  f32x4_t acc[XF][F];
#pragma unroll
  for (int i = 0; i < XF; ++i)
#pragma unroll
    for (int f = 0; f < F; ++f) acc[i][f] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  unsigned char* ring = s_w + team * 2 * C::kTile;
  constexpr int kStep = C::kTK * C::kKW;
  int k0 = k_lo + team * C::kTK;
  load_x(xv[0], k0);
  if constexpr (!WK) {
    if (kEarly) load_w(k0, 0);
    if (steps > 1) load_x(xv[1], k0 + kStep);
    put_w(ring, k0);
    __syncthreads();
  } else if (steps > 1) {
    load_x(xv[1], k0 + kStep);
  }
  // k-contiguous matrices: fragments from memory, a slice ahead while they fit the registers
  constexpr bool kWAhead = WK && F * kQ * (int)sizeof(T) <= 16;
  RowVec<T, 8, MODE> wd[WK ? kQ : 1][WK ? F : 1];
  const auto load_wd = [&](int k) {
    if constexpr (WK)
#pragma unroll
      for (int s = 0; s < kQ; ++s)
#pragma unroll
        for (int f = 0; f < F; ++f) wd[s][f].load(we + (int64_t)min(16 * f + ci, R - 1) * K, k + 32 * s + 8 * q, k_hi);
  };
  if (kWAhead) load_wd(k0);
  const auto slice = [&](int step, X (&v)[XF][kQ]) {
    if (WK && !kWAhead) load_wd(k0);
    Frag xf[XF][kQ];
#pragma unroll
    for (int i = 0; i < XF; ++i)
#pragma unroll
      for (int s = 0; s < kQ; ++s) {
        v[i][s].fix(k0 + 32 * s + 8 * q, k_hi);
        if (!there[i]) v[i][s].zero();
        xf[i][s] = frag_of(v[i][s]);
      }
    const bool more = step + 1 < steps;
    if constexpr (!WK)
      if (kEarly && more) load_w(k0 + kStep, 0);
    if (step + 2 < steps) load_x(v, k0 + 2 * kStep);
    const unsigned char* t = ring + (step & 1) * C::kTile;
#pragma unroll
    for (int s = 0; s < kQ; ++s)
#pragma unroll
      for (int f = 0; f < F; ++f) {
        Frag wf;
        if constexpr (WK) {
          wd[s][f].fix(k0 + 32 * s + 8 * q, k_hi);
          wf = frag_of(wd[s][f]);  // ranks past R repeat the last one; they are not stored
          if (kWAhead && more)
            wd[s][f].load(we + (int64_t)min(16 * f + ci, R - 1) * K, k0 + kStep + 32 * s + 8 * q, k_hi);
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
    if constexpr (!WK) {
      if (!more) return;
      put_w(ring + ((step + 1) & 1) * C::kTile, k0 + kStep);
      __syncthreads();
    }
  };
  for (int step = 0; step < steps; step += 2) {
    slice(step, xv[0]);
    k0 += kStep;
    if (step + 1 < steps) slice(step + 1, xv[1]);
    k0 += kStep;
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
  // rows of part hold Rp ranks, those past R zeros, so that their readers need no ends
  const int Rp = padded(R);
  float* dst = part + (int64_t)blockIdx.y * c.M * Rp;
#pragma unroll
  for (int i = 0; i < XF; ++i) {
    const int m = (rw * XF + i) * 16 + ci;
    if (m >= tile.rows) continue;
    float* row = dst + (int64_t)(tile.row0 + m) * Rp;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int j = 16 * f + 4 * q;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (j + r >= R) acc[i][f][r] = 0.f;
        else if (exact != nullptr) exact[(int64_t)(tile.row0 + m) * R + j + r] = acc[i][f][r];
      }
      if (j < Rp) *reinterpret_cast<f32x4_t*>(row + j) = acc[i][f];
    }
  }
}

// ------------------------------------------------------------------ partial sums

// u[r,j] = s sum_p part[p][r][j] (s the adapter's scale, or 1), rows of `pitch_in`
// ranks, to out (M,R), to rows (M,Rp), and transposed to tr, as grad_kernel reads it:
// (terms,R16,pitch) bf16 terms, two or three, or (R16,pitch) binary32, ranks past R
// zeros; each may be null. Rows of no adapter are zeros in tr and stay as they were
// elsewhere. A block takes 32 grouped rows; blockIdx.y selects one of two such jobs.
struct PackJob {
  const float* part;
  int parts, pitch_in;
  bool scaled;
  float* out;
  float* rows;
  void* tr;
};
constexpr int kPackRows = 32;

template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(LoraCall c, PackJob j0, PackJob j1, int64_t pitch, int terms) {
  __shared__ float s_u[kPackRows * 129];
  __shared__ float s_scale[kPackRows];
  __shared__ int s_off[257];
  const PackJob job = blockIdx.y ? j1 : j0;
  const int r0 = blockIdx.x * kPackRows, R = c.R, R16 = (R + 15) & ~15;
  const int rows = min(kPackRows, c.M - r0);
  for (int i = threadIdx.x; i <= c.e; i += 256) s_off[i] = min(max(c.offsets[i], 0), c.M);
  __syncthreads();
  const int live = min(rows, s_off[c.e] - r0);  // rows of some adapter
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
  // 4 ranks to a thread and step
  const int per = R16 / 4;
  const int64_t slab = (int64_t)c.M * job.pitch_in;
  for (int i = threadIdx.x; i < kPackRows * per; i += 256) {
    const int r = i / per, j = i % per * 4;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < live && j < R) {
      const float* p = job.part + (int64_t)(r0 + r) * job.pitch_in;
#pragma unroll 8
      for (int k = 0; k < job.parts; ++k) {
        // u itself may have rows of any length
        const float* row = p + k * slab;
#pragma unroll
        for (int t = 0; t < 4; ++t) a[t] += row[min(j + t, job.pitch_in - 1)];
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) a[t] = j + t < R ? a[t] * s_scale[r] : 0.f;
      if (job.out != nullptr)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (j + t < R) job.out[(int64_t)(r0 + r) * R + j + t] = a[t];
    }
    // all of a row's padded(R) ranks, those past R zeros: their readers take them all
    if (job.rows != nullptr && r < live && j < padded(R))
      *reinterpret_cast<f32x4_t*>(job.rows + (int64_t)(r0 + r) * padded(R) + j) = (f32x4_t){a[0], a[1], a[2], a[3]};
#pragma unroll
    for (int t = 0; t < 4; ++t) s_u[r * (R16 + 1) + j + t] = a[t];
  }
  if (job.tr == nullptr) return;
  __syncthreads();
  for (int i = threadIdx.x; i < R16 * (kPackRows / 2); i += 256) {
    const int j = i / (kPackRows / 2), r = i % (kPackRows / 2) * 2;  // rows r, r + 1 of rank j; pitch holds whole blocks
    float u0 = s_u[r * (R16 + 1) + j], u1 = s_u[(r + 1) * (R16 + 1) + j];
    const int64_t at = (int64_t)j * pitch + r0 + r;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float2*>((float*)job.tr + at) = make_float2(u0, u1);
    } else {
      const uint32_t hi = upper_terms(u0, u1), lo = pack_bf16x2(u0, u1);
      *reinterpret_cast<uint32_t*>((bf16_t*)job.tr + at) = hi;
      *reinterpret_cast<uint32_t*>((bf16_t*)job.tr + R16 * pitch + at) = lo;
      if (terms > 2)  // what is left has 8 bits at most
        *reinterpret_cast<uint32_t*>((bf16_t*)job.tr + 2 * R16 * pitch + at) =
            pack_bf16x2(u0 - __uint_as_float(lo << 16), u1 - __uint_as_float(lo & 0xffff0000u));
    }
  }
}

// ------------------------------------------------------------------ rows times (R,N)

constexpr int kUpCols = 256;  // columns of a tile, 64 to a wave
constexpr int kUpRows = 64;   // rows: few enough that one block's start overlaps another's stream
                              // (8192 x 4096, rank 16: 42 us, tiles of 256 rows with the next 64
                              // ahead 51; since then 35 by other steps)

__device__ __forceinline__ void swap16(float& a, float& b) {  // odd rows of 16 lanes of a with even ones of b
  const u32x2_t s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(s.x);
  b = __uint_as_float(s.y);
}
__device__ __forceinline__ void swap32(float& a, float& b) {  // the upper half of a with the lower one of b
  const u32x2_t s = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(s.x);
  b = __uint_as_float(s.y);
}
// Piece p of row q of 16 lanes, number 2q + p (4q + p), to piece p' of row q', the same
// number being 4p' + q'.
__device__ __forceinline__ void across(float (&o)[2][8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    swap16(o[0][k], o[1][k]);
    swap32(o[0][k], o[1][k]);
  }
}
__device__ __forceinline__ void across(float (&o)[4][4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    swap16(o[0][k], o[1][k]);
    swap16(o[2][k], o[3][k]);
    swap32(o[0][k], o[2][k]);
    swap32(o[1][k], o[3][k]);
  }
}

// Base, or zeros, in those of a block's kFillRows rows that are not listed: a wave per
// four of them.
template <typename T, int V, int MODE>
__device__ __forceinline__ void fill_rows(const LoraCall& c, int block, int N, const T* base, T* out) {
  constexpr int kRows = kFillRows / 4;
  const int t0 = block * kFillRows + (int)(threadIdx.x / kWave) * kRows, lane = threadIdx.x % kWave;
  const bool gone = lane < kRows && t0 + lane < c.T && !is_listed(c, min(t0 + lane, c.T - 1));
  for (uint64_t left = __ballot(gone); left != 0; left &= left - 1) {
    const int64_t at = (int64_t)(t0 + __builtin_ctzll(left)) * N;
    for (int j = lane * V; j < N; j += 4 * kWave * V) {
      RowVec<T, V, MODE> v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (base != nullptr) v[i].load(base + at, j + i * kWave * V, N);
        else v[i].zero();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i].fix(j + i * kWave * V, N);
        v[i].store(out + at, j + i * kWave * V, N);
      }
    }
  }
}

// WS steps of 32 ranks; WS = 0: up to 16 ranks, the upper and lower
// terms of u side by side in one step (bf16). In a step lane (i, q) holds 8 ranks of
// columns 4i .. 4i+3 of the wave's 64, MFMA f taking column 4i + f as its row i:
// acc[f][r] of lane (row ci, q) is column 16q + 4r + f.
// Over 64 ranks three blocks of a CU are asked for, as the compiler takes registers for
// two (4096 rows 4096 <-> 1024, rank 128, the whole way back: 157 us and 163).
template <typename T, int WS, bool WK, int MODE, bool R8>
__global__ __launch_bounds__(256, sizeof(T) == 2 && WS == 4 && R8 ? 3 : 0)
void up_kernel(LoraCall c, const float* __restrict__ u, int parts, bool scaled, const T* __restrict__ w, int N,
               const T* base, T* out, int blocks) {
  typedef typename Frag8<T>::Type Frag;
  constexpr int kV = 16 / (int)sizeof(T), kP = 16 / kV;  // a lane's 16 columns in pieces of 16 bytes
  typedef RowVec<T, kV, MODE> Y;
  if ((int)blockIdx.x >= blocks) {  // blocks beside the tiles': rows that nobody lists
    fill_rows<T, kV, MODE>(c, blockIdx.x - blocks, N, base, out);
    return;
  }
  constexpr int kS = WS > 0 ? WS : 1, kRF = kUpRows / 16;
  // u's rows as operands: each is added up, scaled and split once for the block's four
  // waves, and read from LDS, so that no load of the loop waits behind its stores (both
  // count on one counter, in order: 8192 x 4096, rank 16 took 43 to 61 us with u from
  // memory, 42 from LDS)
  constexpr int kLo = WS > 0 ? 64 * kS : 32;  // bytes from a row's upper terms to its lower ones
  constexpr int kPitch = 2 * kLo + 16;  // two bf16 terms or one binary32 value a rank, and 16 bytes of padding
  __shared__ __attribute__((aligned(16))) unsigned char s_u[kUpRows * kPitch];
  __shared__ int s_off[257], s_pre[257];
  load_tile_prefix<kUpRows>(c.offsets, c.e, c.M, s_off, s_pre);
  const int ntn = cdiv(N, kUpCols);
  const int total = s_pre[c.e] * ntn;
  // then rows of no adapter, where they are copied
  const int rest = base == out ? 0 : (c.M - s_off[c.e] + kUpRows - 1) / kUpRows * ntn;
  int L;
  if (!xcd_run(blockIdx.x, total + rest, L)) return;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, ci = lane & 15, q = lane >> 4;
  const int R = c.R, Rp = padded(R);
  Tile tile;
  bool idle = false;
  if (L < total) {
    tile_of<kUpRows, kUpCols, 1>(s_off, s_pre, c.e, ntn, L, tile);
  } else {
    // base, or zeros
    L -= total;
    tile.row0 = s_off[c.e] + L / ntn * kUpRows;
    tile.rows = min(kUpRows, c.M - tile.row0);
    tile.n0 = L % ntn * kUpCols;
    tile.ex = 0;
    idle = true;
  }
  const int n0 = tile.n0 + wave * 64;  // past N for the last tile's last waves
  // Pieces move between the four lanes of a row until its accesses are side by side:
  // lane q's pieces kP q + p become p * 4 + q.
  const auto col = [&](int p) { return n0 + (p * 4 + q) * kV; };
  // base's rows first: the longest way
  int t[kRF];
  Y bs[kRF][kP];
#pragma unroll
  for (int i = 0; i < kRF; ++i) t[i] = row_entry(c, tile.row0 + min(16 * i + ci, tile.rows - 1));
#pragma unroll
  for (int i = 0; i < kRF; ++i) {
    const int m = 16 * i + ci;
    t[i] = m < tile.rows ? row_of(c, tile.row0 + m, t[i]) : -1;
  }
  if (base != nullptr)
#pragma unroll
    for (int i = 0; i < kRF; ++i)
#pragma unroll
      for (int p = 0; p < kP; ++p) bs[i][p].load(base + (int64_t)max(t[i], 0) * N, col(p), N);
  Frag wf[kS][4];
  if (!idle) {
    const T* we = w + (int64_t)tile.ex * R * N;
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      const int j0 = WS > 0 ? 32 * s + 8 * q : 8 * (q & 1);
      if constexpr (WK) {
        Ranks<T, R8> v[4];
        Ranks<T, R8>::load(v, R, [&](int f, const T*& row, int& j) {
          row = we + (int64_t)min(n0 + 4 * ci + f, N - 1) * R;  // past N the last column again; not stored
          j = j0;
        });
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          v[f].fix(j0, R);
          wf[s][f] = __builtin_bit_cast(Frag, v[f].x.w);
        }
      } else {
        RowVec<T, 4, MODE> in[8];
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
  if (!idle) {
    const float scale = scaled && c.scale != nullptr ? c.scale[tile.ex] : 1.f;
    const int64_t slab = (int64_t)c.M * Rp;
    constexpr int kPer = WS > 0 ? 8 * kS : 4;  // runs of 4 ranks
    for (int i = threadIdx.x; i < tile.rows * kPer; i += 256) {
      const int r = i / kPer, j = i % kPer * 4;
      f32x4_t a = {0.f, 0.f, 0.f, 0.f};
      if (j < Rp) {
        const f32x4_t* p = reinterpret_cast<const f32x4_t*>(u + (int64_t)(tile.row0 + r) * Rp + j);
#pragma unroll 8
        for (int k = 0; k < parts; ++k) a += p[k * (slab / 4)];
      }
      unsigned char* row = s_u + r * kPitch;
      if constexpr (sizeof(T) == 2) {
        uint2 hi, lo;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x = a[2 * h] * scale, y = a[2 * h + 1] * scale;
          (h ? hi.y : hi.x) = upper_terms(x, y);
          (h ? lo.y : lo.x) = pack_bf16x2(x, y);
        }
        *reinterpret_cast<uint2*>(row + j * 2) = hi;
        *reinterpret_cast<uint2*>(row + kLo + j * 2) = lo;
      } else {
        *reinterpret_cast<f32x4_t*>(row + j * 4) = a * scale;
      }
    }
  }
  __syncthreads();
  if (n0 >= N) return;
#pragma unroll
  for (int i = 0; i < kRF; ++i) {
    f32x4_t acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    if (!idle && 16 * i < tile.rows) {
      const unsigned char* row = s_u + (16 * i + ci) * kPitch;
#pragma unroll
      for (int s = 0; s < kS; ++s) {
        if constexpr (sizeof(T) == 2) {
          // up to 16 ranks: the lower two lane rows take the upper terms, the others the lower ones
          const Frag x = *reinterpret_cast<const Frag*>(row + 64 * s + 16 * q);
          if constexpr (WS > 0) {
            const Frag lo = *reinterpret_cast<const Frag*>(row + kLo + 64 * s + 16 * q);
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[f] = mma(wf[s][f], lo, acc[f]);
          }
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[f] = mma(wf[s][f], x, acc[f]);
        } else {
          // up to 16 ranks: the upper lane rows hold the same ranks again
          Frag x;
          const f32x4_t* p = reinterpret_cast<const f32x4_t*>(row + (WS > 0 ? 128 * s + 32 * q : 32 * (q & 1)));
          const f32x4_t a = p[0], b = p[1];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x.v[k] = WS > 0 || q < 2 ? a[k] : 0.f;
            x.v[4 + k] = WS > 0 || q < 2 ? b[k] : 0.f;
          }
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[f] = mma(wf[s][f], x, acc[f]);
        }
      }
    }
    float o[kP][kV];
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
      for (int k = 0; k < kV; ++k) o[p][k] = acc[k & 3][(p * kV + k) >> 2];
    across(o);
    if (base != nullptr) {
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        float v[kV];
        bs[i][p].get(v, col(p), N);
#pragma unroll
        for (int k = 0; k < kV; ++k) o[p][k] += v[k];
      }
    }
    if (t[i] >= 0)
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        Y y;
        y.put(o[p]);
        y.store(out + (int64_t)t[i] * N, col(p), N);
      }
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
// its rows, 32 rows to a wave and step; the waves' sums meet in LDS. TERMS: of v (bf16).
template <typename T, int F, int TERMS, int MODE>
__global__ __launch_bounds__(256) void grad_kernel(LoraCall c, GradSide a, GradSide b, int tiles_a, int tiles_b,
                                                   int64_t pitch, int split, moe_dtype out_dt) {
  typedef typename Frag8<T>::Type Frag;
  constexpr int CV = 16 / (int)sizeof(T), kCols = CV * 16;
  __shared__ float s_acc[3 * F * kWave * 4 * CV];
  // column tiles of one adapter and matrix side by side, then the other ranks, then
  // the other stretches of rows
  const int all = (tiles_a + tiles_b) * c.e, rank_tiles = cdiv((c.R + 15) / 16, F);
  int L;
  if (!xcd_run(blockIdx.x, all * rank_tiles * split, L)) return;
  const int part_of = L / (all * rank_tiles), rank_tile = L / all % rank_tiles;
  L %= all;
  const bool second = L >= tiles_a * c.e;
  if (second) L -= tiles_a * c.e;
  const int tiles = second ? tiles_b : tiles_a;
  const int C = second ? b.C : a.C;
  const T* y = (const T*)(second ? b.y : a.y);
  const T* vt = (const T*)(second ? b.vt : a.vt);
  const bool by_rank = second ? b.by_rank : a.by_rank;
  const int ex = L / tiles, n0 = L % tiles * kCols;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, ci = lane & 15, q = lane >> 4;
  const int R = c.R, R16 = (R + 15) & ~15, j0 = rank_tile * 16 * F;
  const int lo = min(max(c.offsets[ex], 0), c.M), hi = min(max(c.offsets[ex + 1], 0), c.M);
  const int len = max(hi - lo, 0), per = cdiv(cdiv(len, split), 128) * 128;
  const int r_lo = lo + part_of * per, r_hi = min(hi, r_lo + per);
  f32x4_t acc[CV][F];
#pragma unroll
  for (int v = 0; v < CV; ++v)
#pragma unroll
    for (int f = 0; f < F; ++f) acc[v][f] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  // Step by step: the row numbers two steps ahead, rows and v one step ahead of the
  // products.
  typedef RowVec<T, CV, MODE, MODE == kWhole> X;
  constexpr int kTerms = TERMS;
  X x[8];
  RowVec<T, 8, kLoose> d[F][kTerms];
  int t[8], entry[8];
  const int nc = n0 + CV * ci;
  const auto load_rows = [&](int r8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) entry[k] = row_entry(c, min(r8 + k, r_hi - 1));
  };
  const auto use_rows = [&](int r8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = r8 + k < r_hi ? row_of(c, r8 + k, entry[k]) : -1;
  };
  const auto load = [&](int r8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k].load(y + (int64_t)max(t[k], 0) * C, nc, C);
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int term = 0; term < kTerms; ++term) {
        const int j = min(j0 + 16 * f + ci, R16 - 1);
        d[f][term].load(vt + ((int64_t)term * R16 + j) * pitch, min(r8, r_hi - 1), (int)pitch);
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
        d[f][term].fix(min(r8, r_hi - 1), (int)pitch);
        if (r8 + 8 > r_hi)  // rows of the next adapter, or of none
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (r8 + k >= r_hi) d[f][term].set(k, T(0));
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
  const int64_t base = ((int64_t)(part != nullptr ? part_of * c.e : 0) + ex) * C * R;
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

// Rows of a down tile, 128 or 16 (a block's waves then share K). 16 where the adapters
// have fewer than 32 rows each on average (128 adapters of 16 rows, 4096 -> 4096, rank 16:
// 30 us against 33) and where all have at most 512, as 128 leave the GPU idle (512 rows,
// 4096 -> 4096: rank 16 13 us against 17, rank 128 28 against 34; 1024 rows, rank 64 31
// against 29). Matrices whose k rows are contiguous (wk) are read as fragments without
// LDS, which more waves of fewer rows hide better up to 2048 rows (the whole way back,
// 4 x 512 rows 2048 -> 2048: rank 16 37 us against 40, rank 128 91 against 101; 2 x 2048
// rows 4096 -> 4096, rank 64 122 against 119). K is split until there are about two
// blocks per CU, in slices of at least 512 (4096 -> 4096, 512 rows, rank 64: 18 us, slices
// of 1024 22, of 256 35).
struct DownPlan {
  bool small;
  int tiles, split, range;
};
DownPlan down_plan(int e, int M, int K, bool wk) {
  DownPlan p;
  p.small = M < 32 * e || M <= (wk ? 2048 : 512) || K < 8;
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
void go_down(const LoraCall& c, const DownPlan& p, const void* x, const void* w, int K, float* part, float* exact,
             hipStream_t s) {
  // a row of blocks more, at least one per kMarkRows rows; among the tiles' they would
  // take their places on the CUs (8192 rows 7168 -> 2048, rank 64: 34 us, and 50 so)
  const dim3 grid(p.tiles, p.split + (c.listed != nullptr ? 1 : 0));
  const auto go = [&](auto rw, auto mode, auto r8) {
    hipLaunchKernelGGL((down_kernel<T, F, rw(), rw() == 1 ? 1 : 2, WK, mode(), r8()>), grid, dim3(256), 0, s, c,
                       (const T*)x, (const T*)w, K, p.split, p.range, part, exact);
  };
  const auto by_width = [&](auto rw) {
    with_mode(row_mode(K, 8), [&](auto mode) {
      if constexpr (mode() != kNarrow || rw() == 1) {
        // k-contiguous matrices have no rows of ranks
        if (WK || c.R % 8 != 0) go(rw, mode, std::false_type{});
        else if constexpr (!WK) go(rw, mode, std::true_type{});
      }
    });
  };
  if (p.small) by_width(std::integral_constant<int, 1>{});
  else by_width(std::integral_constant<int, 4>{});
}

template <typename T, bool WK>
void launch_down(const LoraCall& c, const DownPlan& p, const void* x, const void* w, int K, float* part,
                 float* exact, hipStream_t s) {
  switch (frags_of(c.R)) {
    case 1: return go_down<T, 1, WK>(c, p, x, w, K, part, exact, s);
    case 2: return go_down<T, 2, WK>(c, p, x, w, K, part, exact, s);
    case 4: return go_down<T, 4, WK>(c, p, x, w, K, part, exact, s);
    default: return go_down<T, 8, WK>(c, p, x, w, K, part, exact, s);
  }
}

template <typename T, bool WK>
void launch_up(const LoraCall& c, const float* u, int parts, bool scaled, const void* w, int N, const void* base,
               void* out, hipStream_t s) {
  const auto go = [&](auto ws, auto mode, auto r8) {
    // the adapters' tiles, and one more of rows of no adapter than whole tiles hold
    const int64_t most = (int64_t)(cdiv(c.M, kUpRows) + (c.e < c.M ? c.e : c.M) + 1) * cdiv(N, kUpCols);
    const int blocks = (int)((most + 7) & ~7ll);
    const dim3 grid((unsigned)blocks + (c.listed != nullptr ? cdiv(c.T, kFillRows) : 0));
    hipLaunchKernelGGL((up_kernel<T, ws(), WK, mode(), r8()>), grid, dim3(256), 0, s, c, u, parts, scaled, (const T*)w, N,
                       (const T*)base, (T*)out, blocks);
  };
  const auto by_width = [&](auto ws) {
    with_mode(row_mode(N, 8), [&](auto mode) {
      if (!WK || c.R % 8 != 0) go(ws, mode, std::false_type{});
      else if constexpr (WK) go(ws, mode, std::true_type{});
    });
  };
  if (c.R <= 16) by_width(std::integral_constant<int, 0>{});
  else if (c.R <= 32) by_width(std::integral_constant<int, 1>{});
  else if (c.R <= 64) by_width(std::integral_constant<int, 2>{});
  else by_width(std::integral_constant<int, 4>{});
}

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

struct FwdWs {
  size_t part, u, listed, total;
};
// The up tiles of a row read its partial sums once per 256 columns: worth a launch
// that adds them where there are many of them (8192 rows 7168 -> 2048, 7 parts: rank 64,
// 3.7 million sums, 62 us against 66; rank 32, 1.8 million, 49 against 47; 2048 rows
// 4096 -> 2048 of rank 64, 8 parts, 36 against 27).
bool pack_first(const DownPlan& p, int M, int R) { return p.split > 1 && (int64_t)M * R * p.split > 3 << 20; }
FwdWs fwd_ws(int e, int M, int H, int R) {
  const DownPlan p = down_plan(e, M, H, false);
  FwdWs w;
  w.part = 0;
  w.u = round256((size_t)p.split * M * padded(R) * 4);
  w.listed = w.u + (pack_first(p, M, R) ? round256((size_t)M * padded(R) * 4) : 0);
  w.total = w.listed + round256((size_t)M * 4);
  return w;
}

struct BwdWs {
  size_t part, du, dut, ut, ga, gb, listed, total;
  int64_t pitch;
  int split;
};
// Rows of each adapter are split where the columns' blocks are fewer than one per CU,
// into stretches of at least 256 rows on average (8192 rows, 1024 -> 1024, rank 16, 16
// blocks: 42 us in 16 stretches, 47 in 8, 114 in one), and, so that an adapter of many
// rows does not end alone, up to four per CU while a stretch's sums are an eighth of its
// rows' bytes (4 uneven adapters of 8192 rows, 4096 -> 4096, 256 blocks: rank 16 103 us in
// four, 110 in one; rank 64, where they are half, 253 and 189), 256 rows or more again at
// ranks below 8 (60000 rows 64 -> 64, rank 2: 59 us, 66 in 512 stretches).
BwdWs bwd_ws(int es, int e, int M, int H, int N, int R) {
  const DownPlan p = down_plan(e, M, N, true);
  BwdWs w;
  const int R16 = (R + 15) & ~15, cols = 256 / es;
  w.pitch = (M + 63) / 64 * 64;
  w.part = 0;
  size_t o = round256((size_t)p.split * M * padded(R) * 4);
  w.du = o; o += round256((size_t)M * padded(R) * 4);
  const size_t tr = round256((size_t)R16 * w.pitch * (es == 2 ? 6 : 4));  // three bf16 terms, or binary32
  w.dut = o; o += tr;
  w.ut = o; o += tr;
  const int blocks = (cdiv(H, cols) + cdiv(N, cols)) * e * cdiv(R16, es == 2 ? 32 : 64);
  const auto low = [](int a, int b) { return a < b ? a : b; };
  const int fill = low(256 / blocks, M / e / 256), even = low(1024 / blocks, M / e / (R < 8 ? 256 : 32 * R));
  const int split = fill > even ? fill : even;
  w.split = split < 1 ? 1 : split;
  w.ga = o; o += w.split > 1 ? round256((size_t)w.split * e * H * R * 4) : 0;
  w.gb = o; o += w.split > 1 ? round256((size_t)w.split * e * R * N * 4) : 0;
  w.listed = o; o += round256((size_t)M * 4);
  w.total = o;
  return w;
}

template <typename T>
moe_status run_fwd(LoraCall c, const void* x, const void* base, const void* a, const void* b, float* u_out, void* out,
                   unsigned char* ws, hipStream_t s) {
  const DownPlan p = down_plan(c.e, c.M, c.H, false);
  const FwdWs w = fwd_ws(c.e, c.M, c.H, c.R);
  if (c.fill) c.listed = (int32_t*)(ws + w.listed);
  const float* u = (float*)(ws + w.part);
  launch_down<T, false>(c, p, x, a, c.H, (float*)(ws + w.part), p.split == 1 ? u_out : nullptr, s);
  int parts = p.split;
  const bool first = pack_first(p, c.M, c.R);
  if (first || (u_out != nullptr && p.split > 1)) {
    const PackJob job{u, parts, padded(c.R), false, u_out, first ? (float*)(ws + w.u) : nullptr, nullptr};
    hipLaunchKernelGGL(pack_kernel<T>, dim3(cdiv(c.M, kPackRows)), dim3(256), 0, s, c, job, job, (int64_t)0, 0);
    if (first) {
      u = (float*)(ws + w.u);
      parts = 1;
    }
  }
  launch_up<T, false>(c, u, parts, true, b, c.N, base, out, s);
  return launch_status();
}

template <typename T>
moe_status run_bwd(LoraCall c, const void* dout, const void* x, const float* u, const void* a, const void* b,
                   const void* dx_base, void* dx, void* da, void* db, moe_dtype dw_dt, unsigned char* ws,
                   hipStream_t s) {
  const BwdWs w = bwd_ws(sizeof(T), c.e, c.M, c.H, c.N, c.R);
  float* part = (float*)(ws + w.part);
  float* du = (float*)(ws + w.du);
  if (c.fill && dx != nullptr) c.listed = (int32_t*)(ws + w.listed);
  const bool three = sizeof(T) == 2 && dw_dt == MOE_F32;
  if (c.M > 0) {
    // du, and transposed what the weight gradients multiply with
    const bool need = dx != nullptr || da != nullptr;
    const DownPlan p = down_plan(c.e, c.M, c.N, true);
    if (need) launch_down<T, true>(c, p, dout, b, c.N, part, nullptr, s);
    const PackJob of_du{part, p.split, padded(c.R), true, nullptr, du, da != nullptr ? (void*)(ws + w.dut) : nullptr};
    const PackJob of_u{u, 1, c.R, false, nullptr, nullptr, (void*)(ws + w.ut)};
    hipLaunchKernelGGL(pack_kernel<T>, dim3(cdiv(c.M, kPackRows), need && db != nullptr ? 2 : 1), dim3(256), 0, s, c,
                       need ? of_du : of_u, of_u, w.pitch, three ? 3 : 2);
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
  const dim3 grid((unsigned)(((int64_t)(ta + tb) * c.e * cdiv((c.R + 15) / 16, F) * w.split + 7) / 8 * 8));
  const int ma = row_mode(c.H, 16 / sizeof(T)), mb = row_mode(c.N, 16 / sizeof(T));
  const auto go = [&](auto f, auto terms) {
    with_mode(ma > mb ? ma : mb, [&](auto mode) {
      hipLaunchKernelGGL((grad_kernel<T, f(), terms(), mode()>), grid, dim3(256), 0, s, c, ga, gb, ta, tb, w.pitch,
                         w.split, dw_dt);
    });
  };
  const auto by_type = [&](auto f) {
    if constexpr (sizeof(T) == 4) go(f, std::integral_constant<int, 1>{});
    else if (three) go(f, std::integral_constant<int, 3>{});
    else go(f, std::integral_constant<int, 2>{});
  };
  if (F == 1) by_type(std::integral_constant<int, 1>{});
  else if (F == 2 || most == 2) by_type(std::integral_constant<int, 2>{});
  else by_type(std::integral_constant<int, most>{});
  if (w.split > 1) {
    const int64_t na = da != nullptr ? (int64_t)c.e * c.H * c.R : 0, nb = db != nullptr ? (int64_t)c.e * c.R * c.N : 0;
    hipLaunchKernelGGL(grad_finish_kernel, dim3((unsigned)cdiv64(na + nb, 256)), dim3(256), 0, s, ga.part, na, da,
                       gb.part, nb, db, w.split, dw_dt);
  }
  return launch_status();
}

}  // namespace

size_t lora_ws_bytes(int e, int M, int H, int R) {
  return M > 0 ? fwd_ws(e, M, H, R).total : 0;
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
