// mxpp.hip — the grouped MXFP4 product on 256 x 256 and 128 x 128 tiles:
//   out[r,n] = act(sum_b 2^(sa[r,b] - 127) 2^(sw[ex,b,n] - 127) sum_{k in b} a[r,k] w[ex,k,n])
// for rows offsets[ex] <= r < offsets[ex+1], blocks b of 32 k values, E2M1
// values a and w two to a byte along k.
//
// A 16x16x128 block-scaled MFMA takes, in lane 16q + i, the 32 values of scale
// block q of row i, 16 bytes, and on E2M1 it is as long as a 16x16x32 bf16 one
// (16 cycles), so the bytes, fragments and MFMAs of a 128-deep slice are those
// of a 32-deep bf16 slice, and so is the schedule: a 4-slot LDS ring filled by
// LDS DMA three slices ahead.
//  * 256 x 256, 8 waves of 128 rows x 64 columns: between two barriers one half
//    of the tile (waves 0-3 the first 128 rows, waves 4-7 the others) multiplies
//    a whole slice while the other half reads its next fragments and issues its
//    share of the DMA. Slice t is read by the first half between barriers 2t and
//    2t+1 and by the second between 2t+1 and 2t+2; a wave that reads slice u
//    issues its share of slice u+3 into the slot of slice u-1, which both halves
//    have read before barrier 2u. Each wave waits for its share of slice t
//    before barrier 2t. An expert's last row piece of at most 32 rows rides on
//    the tile before it.
//  * 128 x 128, 4 waves of 64 x 64, two blocks per CU, one barrier per slice:
//    after barrier s a wave reads slice s+1's fragments, issues slice s+4 into
//    slice s's slot (whose reads barrier s has waited for) and multiplies s.
// Measured: 65536 rows, 7168 -> 2048, 32 experts 560 to 575 us, 3.4 PFLOP/s, of the
// 8.2 that these MFMAs reach alone. A tile takes 48 us of slices, bound by their
// loads (0.85 us for 37 KB and 0.45 us of MFMAs; 12 percent less without the scale
// loads), and 13 us outside them; nine rounds of tiles stand against 8.3 full ones.
// 1024 rows of 4096 -> 1536 over 128 experts 85 us, 4.9 TB/s of weights.
//
// In LDS, 16-byte chunk c of row r is at position c ^ (r/2)%4 and a fragment one
// 16-byte read. Packed weight row k (two reduction values, 256 or 128 columns)
// holds chunk c at position c ^ wswz(k); a transposing 8-byte read turns eight
// packed rows of 16 columns into a column's 8 bytes per lane (two make a
// fragment), and the 16 rows that 32 lanes touch fall in distinct banks. Row
// scales are words of a slice's four blocks, the four rows 16i + c (i = 0..3) of
// a 64-row group adjacent, so that one 16-byte read fetches a lane's scales of
// four fragments; weight scales keep memory's order, where one word holds
// columns 16j + c (j = 0..3) of a block, byte j being picked by the MFMA.
#include <atomic>
#include <type_traits>

#include "tiles.h"

namespace moe {
namespace {

// Row tiles per group of the tile order (as the other 256 x 256 kernels).
constexpr int kGroup = 8;

template <bool SMALL>
struct MxTile {
  static constexpr int kStages = 4, kBM = SMALL ? 128 : 256, kBN = kBM, kFold = SMALL ? 0 : 32;
  static constexpr int kWaves = SMALL ? 4 : 8, kWavesN = kWaves / 2, kNT = 64 * kWaves;
  static constexpr int kFI = kBM / 32;                // row fragments per wave; four column fragments
  static constexpr int kW = (kBM + kFold) * 64;       // slot: rows (and the tail's), then
  static constexpr int kScX = kW + 64 * kBN;          // 64 packed weight rows, then
  static constexpr int kScW = kScX + (kBM + 2 * kFold) * 4;  // a word per row (whole DMA ops), then
  static constexpr int kStage = kScW + 4 * kBN;       // four blocks' weight scales
  static constexpr int kOutRow = kBN * 2 + 16;
  static constexpr int kOut = (kBM + kFold) * kOutRow;
  static constexpr int kLds = kStages * kStage > kOut ? kStages * kStage : kOut;
  static_assert(kLds <= (SMALL ? 80 : 160) * 1024, "LDS");
  static constexpr int kOps = 5;                      // DMA ops per wave and slice
  __device__ static __forceinline__ int wswz(int k) {
    return SMALL ? (k >> 1 & 3) | ((k >> 4 & 1) << 2) : (k & 7) | ((k >> 4 & 1) << 3);
  }
};

template <bool SMALL>
__global__ __launch_bounds__(SMALL ? 256 : 512) __attribute__((amdgpu_waves_per_eu(2))) void mx_pp_kernel(
    const uint8_t* __restrict__ x, const uint8_t* __restrict__ x_scale, RowMap gx, const uint8_t* __restrict__ w,
    const uint8_t* __restrict__ w_scale, const int32_t* __restrict__ offsets, int e, int A, int Hin, int N, int relu,
    bf16_t* __restrict__ out) {
  typedef MxTile<SMALL> P;
  constexpr int S = P::kStages;
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  Tile t;
  {
    int* s_off = reinterpret_cast<int*>(smem);
    load_tile_prefix<P::kBM, P::kFold>(offsets, e, A, s_off, s_off + 257);
    if (!pick_tile<P::kBM, P::kBN, kGroup, P::kFold>(s_off, s_off + 257, e, N, blockIdx.x, t)) return;
    __syncthreads();  // every lane has its tile before the ring overwrites the prefix
  }
  const bool extra = P::kFold > 0 && t.rows > P::kBM;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / P::kWavesN, wn = wave % P::kWavesN;
  const int ci = lane & 15, kq = lane >> 4;
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  const int nsteps = Hin / 128;
  const uint32_t rowb = (uint32_t)Hin / 2u;
  const bool gat = gx.src != nullptr;

  // ---- DMA sources: two KBs of rows, two of weights and a fifth op per wave
  auto row_of = [&](int row) { return row >= t.rows ? -1 : gat ? gather_src(gx, t.row0 + row) : row; };
  const u32x4_t xsrd = make_srd(x + (gat ? 0 : (int64_t)t.row0 * rowb), (uint32_t)(gat ? gx.rows : t.rows) * rowb);
  const u32x4_t wsrd = make_srd(w + (int64_t)t.ex * rowb * N, rowb * (uint32_t)N);
  auto x_off = [&](int kb) {  // byte kb of a slot's rows
    const int row = kb >> 6, src = row_of(row);
    return (src >= 0 ? (uint32_t)src * rowb : kOOB) + (uint32_t)(((kb >> 4 & 3) ^ (row >> 1 & 3)) * 16);
  };
  uint32_t x_voff[2], w_voff[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int kb = (wave * 2 + q) * 1024 + lane * 16;
    x_voff[q] = x_off(kb);
    const int k = kb / P::kBN, col = t.n0 + (((kb % P::kBN) >> 4) ^ P::wswz(k)) * 16;
    w_voff[q] = (uint32_t)k * (uint32_t)N + (uint32_t)col + (col < N ? 0u : kOOB);
  }
  // The fifth op. 256 x 256: roles 0-3 64 rows' scales each, 4 the tail rows'
  // scales, 5 the weight scales, 6 and 7 the tail rows (out of range without a
  // tail), dealt to the two halves in turn. 128 x 128: waves 0 and 1 64 rows'
  // scales each, 2 and 3 half of the weight scales each.
  const int role = SMALL ? wave : wave >> 2 | (wave & 3) << 1;
  const int n64 = (N + 63) & ~63;
  const int srows = gat ? gx.rows : A;
  const bool row_scales = role < (SMALL ? 2 : 5), w_scales = SMALL ? role >= 2 : role == 5;
  const bool words = SMALL || row_scales;  // 4 bytes per lane, else 16
  const uint8_t* base5;
  uint32_t voff5, lds5, bytes5;
  int64_t stride5;  // bytes per slice, of the row scales per two slices
  if (row_scales) {
    const int row = role < 4 ? 64 * role + 16 * (lane & 3) + (lane >> 2) : P::kBM + lane;
    const int src = role == 4 && lane >= 32 ? -1 : row_of(row);
    voff5 = src >= 0 ? (uint32_t)src * 8u : kOOB;
    lds5 = P::kScX + role * 256;
    base5 = x_scale + (gat ? 0 : (int64_t)t.row0 * 8);
    bytes5 = (uint32_t)(gat ? gx.rows : t.rows) * 8u;
    stride5 = (int64_t)srows * 8;
  } else if (w_scales) {
    const int piece = SMALL ? 64 * (role - 2) + lane : lane;
    const int blk = piece / (SMALL ? 32 : 16), col = t.n0 + (SMALL ? 4 * (piece % 32) : 16 * (piece % 16));
    voff5 = (uint32_t)blk * (uint32_t)n64 + (uint32_t)col + (col < n64 ? 0u : kOOB);
    lds5 = P::kScW + (SMALL ? (role - 2) * 256 : 0);
    base5 = w_scale + (int64_t)t.ex * (Hin / 32) * n64;
    bytes5 = 4u * (uint32_t)n64;
    stride5 = bytes5;
  } else {  // (offsets that are not kOOB stay inside a row as the base moves along it)
    voff5 = x_off(P::kBM * 64 + (role - 6) * 1024 + lane * 16);
    lds5 = P::kBM * 64 + (role - 6) * 1024;
    base5 = x + (gat ? 0 : (int64_t)t.row0 * rowb);
    bytes5 = (uint32_t)(gat ? gx.rows : t.rows) * rowb;
    stride5 = 64;
  }
  // Past-the-end slices are issued too (out-of-range loads write zeros), so
  // every wait count is fixed.
  auto issue = [&](int step) {
    const uint32_t base = lds0 + (step % S) * P::kStage;
    const uint32_t past = step < nsteps ? 0u : kOOB;
    const uint32_t st = step < nsteps ? (uint32_t)step : 0u;
#pragma unroll
    for (int q = 0; q < 2; ++q) dma16(xsrd, (x_voff[q] + st * 64u) | past, base + (wave * 2 + q) * 1024);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      dma16(wsrd, (w_voff[q] + st * 64u * (uint32_t)N) | past, base + P::kW + (wave * 2 + q) * 1024);
    const u32x4_t srd5 = make_srd(base5 + (int64_t)(row_scales ? st >> 1 : st) * stride5, bytes5);
    const uint32_t v5 = (voff5 + (row_scales ? (st & 1u) * 4u : 0u)) | past;
    if (words) dma4(srd5, v5, base + lds5);
    else dma16(srd5, v5, base + lds5);
  };

  // ---- fragments
  const int xoff = (wm * P::kFI * 16 + ci) * 64 + ((kq ^ (ci >> 1 & 3)) << 4);  // of fragment 0, 1 KB apart
  const int mt = P::kBM + wm * 16 + ci;                                        // row of the tail fragment
  const int xoff_t = mt * 64 + ((kq ^ (ci >> 1 & 3)) << 4);
  int woff[4];
  const int wk = 16 * kq + (ci >> 1);  // this lane names 8 bytes of packed rows wk and wk + 8
#pragma unroll
  for (int j = 0; j < 4; ++j) woff[j] = P::kW + wk * P::kBN + (((4 * wn + j) ^ P::wswz(wk)) << 4) + 8 * (ci & 1);
  typedef int i32x2_t __attribute__((ext_vector_type(2)));
  typedef int i32x4_t __attribute__((ext_vector_type(4)));
  struct Frags {
    i32x4_t x[P::kFI], t, w[4];
    uint4 sx[P::kFI / 4];
    uint32_t st, sw;
  };
  auto read_frags = [&](int slice, Frags& f, auto ex_) {
    const unsigned char* st = smem + (slice % S) * P::kStage;
#pragma unroll
    for (int i = 0; i < P::kFI; ++i) f.x[i] = *reinterpret_cast<const i32x4_t*>(st + xoff + i * 1024);
    if (decltype(ex_)::value) f.t = *reinterpret_cast<const i32x4_t*>(st + xoff_t);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      typedef __attribute__((address_space(3))) i32x2_t lds_i32x2;
      const i32x2_t a = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(st + woff[j]));
      const i32x2_t b = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(st + woff[j] + 8 * P::kBN));
      f.w[j] = __builtin_shufflevector(a, b, 0, 1, 2, 3);
    }
#pragma unroll
    for (int h = 0; h < P::kFI / 4; ++h)
      f.sx[h] = *reinterpret_cast<const uint4*>(st + P::kScX + ((wm * (P::kFI / 4) + h) * 64 + 4 * ci) * 4);
    if (decltype(ex_)::value) f.st = *reinterpret_cast<const uint32_t*>(st + P::kScX + mt * 4);
    f.sw = *reinterpret_cast<const uint32_t*>(st + P::kScW + kq * P::kBN + wn * 64 + 4 * ci);
  };
  f32x4_t acc[P::kFI][4], acct[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int i = 0; i < P::kFI; ++i) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    acct[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  }
  auto product = [&](const i32x4_t& xv, uint32_t sx, const Frags& f, f32x4_t (&c)[4]) {
    const i32x8_t xf = __builtin_shufflevector(xv, xv, 0, 1, 2, 3, -1, -1, -1, -1);
    const int s = (int)(sx >> (8 * kq));
    auto one = [&](auto J) {
      constexpr int j = decltype(J)::value;
      const i32x8_t wf = __builtin_shufflevector(f.w[j], f.w[j], 0, 1, 2, 3, -1, -1, -1, -1);
      c[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf, c[j], 4, 4, j, (int)f.sw, 0, s);
    };
    one(std::integral_constant<int, 0>{});
    one(std::integral_constant<int, 1>{});
    one(std::integral_constant<int, 2>{});
    one(std::integral_constant<int, 3>{});
    // keeps the products in their phase: free of side effects, they are else moved behind the next reads
    asm volatile("" : "+v"(c[0]), "+v"(c[1]), "+v"(c[2]), "+v"(c[3]));
  };
  auto multiply = [&](const Frags& f, auto ex_) {
#pragma unroll
    for (int i = 0; i < P::kFI; ++i) {
      const uint4 s4 = f.sx[i >> 2];
      product(f.x[i], (i & 3) == 0 ? s4.x : (i & 3) == 1 ? s4.y : (i & 3) == 2 ? s4.z : s4.w, f, acc[i]);
    }
    if (decltype(ex_)::value) product(f.t, f.st, f, acct);
  };
  const bool active = wm * (P::kBM / 2) < t.rows && t.n0 + wn * 64 < N;
  // The compiler may not move work across these barriers: the phases are the schedule.
  auto bar = [] {
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int kInFlight = (S - 2) * P::kOps;
  auto run = [&](auto ex_) {
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(s);
    wait_vmcnt<kInFlight>();
    bar();  // barrier 0: slice 0 has landed
    Frags f;
    if constexpr (SMALL) {
      Frags g;
      read_frags(0, f, ex_);
      issue(S - 1);
      auto step = [&](int s, const Frags& now, Frags& next) {
        wait_vmcnt<kInFlight>();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        bar();  // slice s+1 has landed; every wave holds its fragments of slice s
        read_frags(s + 1, next, ex_);
        issue(s + S);
        multiply(now, ex_);
      };
      for (int s = 0; s < nsteps; s += 2) {  // Hin is a multiple of 256
        step(s, f, g);
        step(s + 1, g, f);
      }
      return;
    }
    if (wm == 1) bar();
    if (active) {
      read_frags(0, f, ex_);
      issue(S - 1);
      wait_vmcnt<kInFlight>();
      bar();
      for (int s = 0; s < nsteps; ++s) {
        multiply(f, ex_);
        bar();
        read_frags(s + 1, f, ex_);
        issue(s + S);
        wait_vmcnt<kInFlight>();
        bar();
      }
    } else {
      issue(S - 1);
      wait_vmcnt<kInFlight>();
      bar();
      for (int s = 0; s < nsteps; ++s) {
        bar();
        issue(s + S);
        wait_vmcnt<kInFlight>();
        bar();
      }
    }
    if (wm == 0) bar();  // matches the second half's last barrier
  };
  if constexpr (P::kFold > 0) {
    if (extra) run(std::true_type{});
    else run(std::false_type{});
  } else {
    run(std::false_type{});
  }
  wait_vmcnt<0>();  // no DMA may still be landing when the block's LDS is reused
  __syncthreads();

  // ---- epilogue: fragment i's row (kFI: the tail), columns 4 kq .. 4 kq + 3 of column fragment j
  if (active) {
#pragma unroll
    for (int i = 0; i < P::kFI + (P::kFold > 0 ? 1 : 0); ++i) {
      if (i == P::kFI && !extra) continue;  // compile-time i keeps the accumulators in registers
      const int ml = i < P::kFI ? (wm * P::kFI + i) * 16 + ci : mt;
      if (ml >= t.rows) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4_t a = i < P::kFI ? acc[i][j] : acct[j];
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = relu && a[r] < 0.f ? 0.f : a[r];
        *reinterpret_cast<uint2*>(smem + ml * P::kOutRow + (wn * 64 + j * 16 + 4 * kq) * 2) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
    }
  }
  __syncthreads();
  constexpr int kLanes = P::kBN / 8;  // lanes per row
#pragma unroll 1
  for (int idx = tid; idx < t.rows * kLanes; idx += P::kNT) {
    const int row = idx / kLanes, col = idx % kLanes * 8;
    if (t.n0 + col >= N) continue;  // N is a multiple of 16
    *reinterpret_cast<uint4*>(out + (int64_t)(t.row0 + row) * N + t.n0 + col) =
        *reinterpret_cast<const uint4*>(smem + row * P::kOutRow + col * 2);
  }
}

// Estimated time in microseconds, from what the two tile sizes measured over 23
// shapes of 64 to 65536 rows: per slice and per tile outside its loop, with one
// tile per CU (large) or two (small; a CU left with one small tile runs it
// faster). Rows per expert are taken as the average, with half a tile of slack
// for each expert. The tile sizes give the same bits. Measured (large / small):
// 65536 rows, 7168 -> 2048, 32 experts 567 / 668 us; 512 rows, 4096 -> 4096, one
// expert 36 / 16; 2048 rows, 4096 -> 1536, 128 experts 89 / 84; 1024 rows,
// 4096 -> 14336, 8 experts 72 / 91.
double tiles_time(int e, int A, int Hin, int N, bool small, int ncu) {
  const int bm = small ? 128 : 256;
  const int experts = e < A ? e : A, slices = Hin / 128;
  const double tiles = (experts == 1 ? (double)cdiv(A, bm) : (double)A / bm + 0.5 * experts) * cdiv(N, bm);
  const double per = small ? 2.0 * ncu : ncu;
  const double full = (double)(int64_t)(tiles / per), rest = tiles - full * per;
  if (!small) return (full + (rest > 0)) * (0.85 * slices + 10);
  return full * (0.60 * slices + 7) + (rest > ncu ? 0.60 * slices + 7 : rest > 0 ? 0.33 * slices + 6 : 0);
}
bool takes_small(int e, int A, int Hin, int N, int ncu) {
  return tiles_time(e, A, Hin, N, true, ncu) < tiles_time(e, A, Hin, N, false, ncu);
}

template <bool SMALL>
moe_status launch_size(const uint8_t* x, const uint8_t* x_scale, RowMap gx, const uint8_t* w, const uint8_t* w_scale,
                       const int32_t* offsets, int e, int A, int Hin, int N, int relu, bf16_t* out, hipStream_t s) {
  typedef MxTile<SMALL> P;
  static std::atomic<uint64_t> done{0};  // devices on which the kernel may use its LDS
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  if (!(done.load(std::memory_order_relaxed) >> dev & 1)) {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(&mx_pp_kernel<SMALL>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, P::kLds);
    done.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  const int64_t grid = cdiv64((cdiv64(A, P::kBM) + (e < A ? e : A)) * cdiv(N, P::kBN), 8) * 8;
  if (grid > 0x7fffffff) return MOE_ERR_BAD_SHAPE;
  hipLaunchKernelGGL(mx_pp_kernel<SMALL>, dim3((unsigned)grid), dim3(P::kNT), P::kLds, s, x, x_scale, gx, w, w_scale,
                     offsets, e, A, Hin, N, relu, out);
  return launch_status();
}

}  // namespace

moe_status launch_mx_pp(const uint8_t* x, const uint8_t* x_scale, RowMap gx, const uint8_t* w, const uint8_t* w_scale,
                        const int32_t* offsets, int e, int A, int Hin, int N, moe_act act, void* out, hipStream_t s) {
  if (A == 0) return MOE_OK;
  const int relu = act == MOE_ACT_RELU;
  return takes_small(e, A, Hin, N, device_cus())
             ? launch_size<true>(x, x_scale, gx, w, w_scale, offsets, e, A, Hin, N, relu, (bf16_t*)out, s)
             : launch_size<false>(x, x_scale, gx, w, w_scale, offsets, e, A, Hin, N, relu, (bf16_t*)out, s);
}

}  // namespace moe
