// tiles.h — device helpers shared by the grouped kernels: the tile order over
// experts, row gathers, buffer descriptors and LDS DMA.
#pragma once

#include "common.h"

namespace moe {
namespace {

// ------------------------------------------------------------------ helpers

// Expert offsets (clamped to [0, A]) and the running count of row tiles per
// expert, in LDS: s_off[0..e], s_pre[0..e] (s_pre[q] = tiles before expert q).
// Row tiles of an expert with `rows` rows: ceil(rows / BM), except that a
// last piece of at most FOLD rows rides on the tile before it (that tile
// then has BM < rows <= BM + FOLD).
template <int BM, int FOLD>
__device__ __forceinline__ int row_tiles(int rows) {
  const int t = (rows + BM - 1) / BM;
  const int tail = rows - (t - 1) * BM;
  return (FOLD > 0 && t > 1 && tail <= FOLD) ? t - 1 : t;
}

template <int BM, int FOLD = 0>
__device__ __forceinline__ void load_tile_prefix(const int32_t* __restrict__ offsets, int e, int A,
                                                 int* s_off, int* s_pre) {
  for (int q = threadIdx.x; q <= e; q += blockDim.x) {
    int v = offsets[q];
    s_off[q] = v < 0 ? 0 : (v > A ? A : v);
  }
  __syncthreads();
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x;
    // each lane covers 4 consecutive experts (e <= 256)
    int c[4], local = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = lane * 4 + i;
      int rows = q < e ? s_off[q + 1] - s_off[q] : 0;
      rows = rows < 0 ? 0 : rows;
      c[i] = row_tiles<BM, FOLD>(rows);
      local += c[i];
    }
    const int incl = wave_incl_scan(local);
    int run = incl - local;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = lane * 4 + i;
      if (q < e) s_pre[q] = run;
      run += c[i];
    }
    if (lane == kWave - 1) s_pre[e] = incl;  // total row tiles
  }
  __syncthreads();
}

struct Tile {
  int ex, row0, rows, n0;
};

// Source row of grouped row r under a gather (gx.src != nullptr), or -1 when
// the entry's quotient falls outside [0, gx.rows).
__device__ __forceinline__ int gather_src(const RowMap& gx, int r) {
  const int v = gx.src[r];
  const int q = v >= 0 ? v / gx.div : -1;
  return q < gx.rows ? q : -1;
}

// Where grouped row m is stored (row m itself without an output map) and the
// factor it is multiplied by (its gate, else 1); row -1: not stored (a
// destination outside [0, A)).
struct OutRow {
  int64_t row;
  float gate;
};
__device__ __forceinline__ OutRow out_row_of(const RowMap& rm, int64_t m, int d, int A) {
  if (rm.dst == nullptr) return {m, 1.f};
  if (d < 0 || d >= A) return {-1, 0.f};
  return {d, rm.gate != nullptr ? rm.gate[d] : 1.f};
}
__device__ __forceinline__ OutRow out_row(const RowMap& rm, int64_t m, int A) {
  return out_row_of(rm, m, rm.dst != nullptr ? rm.dst[m] : 0, A);
}

// Per-row activation scale of grouped row m (1 without one); a gathered row
// whose index is out of range reads as a zero row, scale 0.
__device__ __forceinline__ float row_scale_of(const RowMap& rm, int m) {
  if (rm.row_scale == nullptr) return 1.f;
  if (rm.src == nullptr) return rm.row_scale[m];
  const int t = gather_src(rm, m);
  return t >= 0 ? rm.row_scale[t] : 0.f;
}

// Tile of logical index L (0 <= L < s_pre[e] * ntn). Inside an expert,
// tiles go in groups of GM row tiles: group-major, then column tile, then
// row tile.
template <int BM, int BN, int GM, int FOLD = 0>
__device__ __forceinline__ void tile_of(const int* s_off, const int* s_pre, int e, int ntn, int L, Tile& t) {
  const int g = L / ntn;  // global row-tile-major position among s_pre[e] row tiles
  // find expert ex with s_pre[ex] <= g < s_pre[ex+1] (binary search, s_pre non-decreasing)
  int lo = 0, hi = e - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_pre[mid] <= g) lo = mid;
    else hi = mid - 1;
  }
  const int ex = lo;
  const int mt = s_pre[ex + 1] - s_pre[ex];
  const int q = L - s_pre[ex] * ntn;  // local index within the expert
  const int grp = q / (GM * ntn);
  const int within = q - grp * GM * ntn;
  const int gsz = min(GM, mt - grp * GM);
  const int nt = within / gsz;
  const int m = grp * GM + within % gsz;
  // every lane computed the same tile: say so, so that tile-derived bases and
  // buffer descriptors live in scalar registers
  t.ex = __builtin_amdgcn_readfirstlane(ex);
  t.row0 = __builtin_amdgcn_readfirstlane(s_off[ex] + m * BM);
  const int left = s_off[ex + 1] - (s_off[ex] + m * BM);  // the last tile takes a folded tail
  t.rows = __builtin_amdgcn_readfirstlane((FOLD > 0 && m == mt - 1) ? left : min(BM, left));
  t.n0 = __builtin_amdgcn_readfirstlane(nt * BN);
}

// Logical tile for this block, or false if the block has no work.
// XCD-aware: block p runs on XCD p % 8; XCD x takes logical tiles
// [x*per, (x+1)*per).
template <int BM, int BN, int GM, int FOLD = 0>
__device__ __forceinline__ bool pick_tile(const int* s_off, const int* s_pre, int e, int N, int p, Tile& t) {
  const int ntn = (N + BN - 1) / BN;
  const int total = s_pre[e] * ntn;
  if (total == 0) return false;
  const int per = (total + 7) / 8;
  const int slot = p >> 3;
  if (slot >= per) return false;
  const int L = (p & 7) * per + slot;
  if (L >= total) return false;
  tile_of<BM, BN, GM, FOLD>(s_off, s_pre, e, ntn, L, t);
  return true;
}

// ------------------------------------------------------------------ LDS DMA helpers
//
// gfx950 LDS DMA: buffer_load_dwordx4 ... lds moves 16 bytes per lane from
// global memory straight into LDS at M0 + 16*lane, with no staging
// registers; out-of-range buffer offsets write zeros. Every DMA instruction
// of the ping-pong kernels fills one contiguous KB of a ring slot; the
// swizzles live in which global bytes each lane fetches.

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));


__device__ __forceinline__ u32x4_t make_srd(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)base;
  u32x4_t r;
  r.x = __builtin_amdgcn_readfirstlane((uint32_t)b);
  r.y = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) & 0xffffu;  // stride 0
  r.z = __builtin_amdgcn_readfirstlane(bytes);                          // loads past it read 0
  r.w = 0x00020000u;                                                    // 32-bit data format
  return r;
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 bytes per lane from buffer offset voff into LDS at lds_base + 16*lane
// (lds_base wave-uniform). The compiler does not see these loads, so the
// kernel waits for them itself with wait_vmcnt.
__device__ __forceinline__ void dma16(u32x4_t srd, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(srd), "s"(lds_base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// 4 bytes per lane from buffer offset voff into LDS at lds_base + 4*lane.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma4(u32x4_t srd, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(srd), "s"(lds_base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Bytes: rows r0..r7 of 8 columns (uint2 each, one byte per column) ->
// 8 columns of 8 rows (uint2 each, one byte per row).
__device__ __forceinline__ void transpose_8x8_u8(const uint2 in[8], uint2 out[8]) {
#pragma unroll
  for (int c = 0; c < 8; c += 2) {
    // byte c and c+1 of each row; rows paired (0,1),(2,3),(4,5),(6,7)
    const int d = c >> 2;        // which dword of the row
    const int b = c & 3;         // byte within it (0 or 2)
    // pair[p] = {r2p[c], r2p+1[c], r2p[c+1], r2p+1[c+1]}
    const uint32_t sel_pair = (uint32_t)(b) | ((uint32_t)(4 + b) << 8) | ((uint32_t)(b + 1) << 16) |
                              ((uint32_t)(5 + b) << 24);
    uint32_t pr[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t lo = d ? in[2 * p].y : in[2 * p].x;
      const uint32_t hi = d ? in[2 * p + 1].y : in[2 * p + 1].x;
      pr[p] = perm_b32(hi, lo, sel_pair);
    }
    // column c: {r0,r1,r2,r3} = lo16(pr0) | lo16(pr1)<<16 ; {r4..r7} from pr2, pr3
    out[c].x = perm_b32(pr[1], pr[0], 0x05040100u);
    out[c].y = perm_b32(pr[3], pr[2], 0x05040100u);
    out[c + 1].x = perm_b32(pr[1], pr[0], 0x07060302u);
    out[c + 1].y = perm_b32(pr[3], pr[2], 0x07060302u);
  }
}

// Where a 16-bit transposing LDS read (ds_read_b64_tr_b16) takes its rows: it
// reads k rows 0-3 and 8-11 (then 4-7 and 12-15) in one pass of 32 lanes, 32
// bytes of each. Stored with their 32-byte units u of k row k at position u ^
// unit_swz(bytes per k row, k), those fall in distinct banks.
__device__ __forceinline__ constexpr int unit_swz(int pitch, int k) {
  return pitch == 64 ? k >> 3 & 1 : pitch == 128 ? (k >> 1 & 1) | ((k >> 3 & 1) << 1) : (k & 3) | ((k >> 3 & 1) << 2);
}

// Compute units of the current device.
int device_cus() {
  static int cus[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (cus[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
    cus[dev] = n;
  }
  return cus[dev];
}

}  // namespace
}  // namespace moe
