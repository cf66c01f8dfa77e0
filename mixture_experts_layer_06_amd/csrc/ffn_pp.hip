// ffn_pp.hip — the products of the gated feed-forward and the gradients (ffn.hip
// states them) on tiles filled by LDS DMA, for rows that start on 16 bytes.
//
// One set of loads and fragments for all three; the reduction is walked in
// slices of 64 bytes per row (32 bf16 values, 16 of binary32) through a 4-slot
// LDS ring, every wave moving 3 or 4 KB of each slice. Tile sizes:
//  * 256 x 256, 8 waves of 128 m x 64 n: the two halves of the tile (waves
//    0-3: m < 128, waves 4-7) run out of phase. Between two barriers one half
//    multiplies a whole slice while the other reads its next fragments and
//    issues its share of the DMA, so each SIMD's matrix pipe is fed by one wave
//    while its partner works on memory. Slice t is read by the first half
//    between barriers 2t and 2t+1 and by the second between 2t+1 and 2t+2; a
//    wave that reads slice u issues its share of slice u+3, which goes to the
//    slot of slice u-1, read by both halves before barrier 2u. Each wave waits
//    for its share of slice t before barrier 2t, leaving those of t+1 and t+2
//    in flight. An expert's last row piece of at most 32 rows rides on the tile
//    before it.
//  * 128 x 128, 4 waves of 64 x 64, two blocks per CU, one barrier per slice:
//    after barrier s a wave reads the fragments of slice s+1, issues slice s+4
//    into the slot of slice s (whose reads barrier s has waited for) and
//    multiplies slice s. Taken where the large tiles are too few for the CUs
//    or too short, and for binary32,
//  * which also has 64 x 128 tiles, three blocks per CU, on the same schedule.
// Measured: bf16 GLU of 8192 rows, 4096 -> 14336, 8 experts 1546 to 1670 us, 1.15
// to 1.24 PFLOP/s (a library product of one such expert's size 1.17); dgrad of the
// same 830 to 900, 1.07 to 1.16, wgrad 1010 to 1090, 0.88 to 0.95. Those are bound by
// the matrix pipe at the clock the power limit leaves (1.6 to 2.1 GHz; pipe busy
// 0.64, 0.51 to 0.60, 0.47 to 0.48), the rest being barriers and the tiles' first slices and
// stores. binary32 is bound by its MFMAs (16x16x4, 32 cycles each): GLU of 8192
// rows, 1024 -> 2048, one expert 534 us, 129 TFLOP/s (library product 153).
//
// Operands sit in LDS as memory has them:
//  * k contiguous (rows x 64 bytes): 16-byte chunk c of row r at position
//    c ^ (r/2)%4; a fragment is one 16-byte read (binary32: values 4q .. 4q+3 of
//    row i in lane 16q + i, MFMA s taking value s of each).
//  * k strided (32 k rows of 512 or 256 bytes, GLU's in two panels of half
//    that): 32-byte unit u of k row k at position u ^ (k%4 + 4 (k/8%2)), in
//    128-byte rows, which alternate between the bank halves, u ^ (k/2%2 + 2
//    (k/8%2)); a fragment is two transposing 8-byte reads. In such a read each 16 lanes name a 4 x 16
//    block (lane 4b+c bytes 8c..8c+7 of row b's 32) and lane l receives column
//    l; lanes 0-31 touch k rows 0-3 and 8-11 (+4 in the second read), which
//    the swizzle spreads over all 64 banks. binary32 (16 k rows of 512 or 256
//    bytes): 64-byte unit u of row k at u ^ k/4%4, four 4-byte reads.
// GLU's n operand holds gate columns and the same number of up columns, a
// wave's four n fragments being two of each, so that one lane ends with g and u
// of the same outputs and multiplies them in registers. In WGRAD the two
// gradients dg and du are adjacent columns of one matrix, as are its outputs.
//
// The output tile goes through LDS so that whole rows are stored.
#include <atomic>

#include "tiles.h"

namespace moe {
namespace {

enum { GLU = 0, DGRAD = 1, WGRAD = 2 };

#include "act.h"

typedef short i16x4_t __attribute__((ext_vector_type(4)));

// Row tiles per group of the tile order (as the other 256 x 256 kernel).
constexpr int kGroup = 8;

// Tile sizes: 256 x 256, 128 x 128, 64 x 128.
enum { LARGE = 0, SMALL = 1, FLAT = 2 };

template <int MODE, typename TO, int SIZE, typename T>
struct PpTile {
  static constexpr int kES = sizeof(T), kSK = 64 / kES;  // bytes of an element, k values of a slice
  static constexpr int kStages = 4, kBM = SIZE == LARGE ? 256 : SIZE == SMALL ? 128 : 64, kFold = MODE == WGRAD || SIZE != LARGE ? 0 : 32;
  static constexpr int kWaves = SIZE == LARGE ? 8 : 4, kWavesN = kWaves / 2, kNT = 64 * kWaves;
  static constexpr int kNR = SIZE == LARGE ? 256 : 128;                         // rows of the n operand
  static constexpr int kBN = MODE == GLU ? kNR / 2 : kNR;  // output columns
  static constexpr int kFI = kBM / 32;                    // m fragments per wave; four n fragments
  static constexpr int kLdsX = (kBM + kFold) * 64;        // == kSK k rows of kBM values without a fold
  static constexpr int kLdsW = kNR * 64;
  static constexpr int kStage = kLdsX + kLdsW;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kXPitch = kBM * kES, kWPitch = kBN * kES;  // bytes of a k row (k strided operands)
  static constexpr int kOutRow = kBN * (int)sizeof(TO) + 16;
  static constexpr int kPasses = sizeof(TO) == 4 && SIZE == LARGE ? 2 : 1;
  // rows staged at a time: all, or (fp32, 256 columns) one wave half's
  static constexpr int kOutRows = kPasses == 2 ? 128 : kBM + kFold;
  static constexpr int kXOps = kBM / 16 / kWaves;            // KBs of x a wave fills per slice; two of w
  static constexpr int kLds = kRing > kOutRows * kOutRow ? kRing : kOutRows * kOutRow;
  // WGRAD gather: k rows a wave fetches per slice, slices per 64 row offsets
  static constexpr int kRW = kSK / kWaves, kSB = 64 / kRW;
  static constexpr int kIdx = MODE == WGRAD ? kWaves * 2 * 256 : 0;  // the offsets, past the rest
  static_assert(kLds + kIdx <= (SIZE == LARGE ? 160 : SIZE == SMALL ? 80 : 53) * 1024, "LDS");
  // Byte of a k row of `pitch` bytes that byte b of row k's place in LDS holds:
  // units of 16 columns are spread so that the reads of a fragment fall in
  // distinct banks (bf16: unit_swz; binary32: a read takes rows 4q + s, q = 0..3).
  static constexpr int kUnit = 16 * kES;
  static __device__ __forceinline__ int swz(int pitch, int k) { return kES == 4 ? k >> 2 & 3 : unit_swz(pitch, k); }
  static __device__ __forceinline__ int source(int pitch, int k, int b) {
    return ((b / kUnit) ^ swz(pitch, k)) * kUnit + b % kUnit;
  }
};

template <int MODE, typename TO, int SIZE, typename T>
__global__ __launch_bounds__(SIZE == LARGE ? 512 : 256)
    __attribute__((amdgpu_waves_per_eu(SIZE == FLAT ? 3 : 2))) void ffn_pp_kernel(FfnCall c) {
  typedef PpTile<MODE, TO, SIZE, T> P;
  constexpr bool kF32 = sizeof(T) == 4;
  static_assert(!kF32 || SIZE != LARGE, "no large binary32 tiles");
  static_assert(MODE != WGRAD || SIZE != FLAT, "gradients of weights have no ragged rows");
  constexpr int S = P::kStages;
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];

  // ---- the tile
  int ex, m0, mrows, n0, r0 = 0, rows_k = 0;
  if (MODE == WGRAD) {
    // Every expert's (and part's) tiles are spread over the 8 XCDs in
    // contiguous runs (experts differ in depth, so whole experts per XCD would
    // not balance), starting at the XCD after the one before's last.
    const int ntm = cdiv(c.Hin, P::kBM), ntn = cdiv(c.npair * c.N, P::kBN);
    const int per = cdiv(ntm * ntn, 8), used = cdiv(ntm * ntn, per);
    const int slot = blockIdx.x >> 3;
    ex = slot / per;
    const uint32_t before = (uint32_t)(blockIdx.y * c.e + ex) * (uint32_t)used;
    const int q = (int)((blockIdx.x - before) & 7u) * per + slot % per;
    if (q >= ntm * ntn) return;
    const int grp = q / (kGroup * ntn), within = q - grp * kGroup * ntn;
    const int gsz = min(kGroup, ntm - grp * kGroup);
    m0 = (grp * kGroup + within % gsz) * P::kBM;
    n0 = within / gsz * P::kBN;
    mrows = min(P::kBM, c.Hin - m0);
    const int a = c.offsets[ex], b = c.offsets[ex + 1];
    r0 = a < 0 ? 0 : a > c.A ? c.A : a;
    rows_k = (b < 0 ? 0 : b > c.A ? c.A : b) - r0;
    if (rows_k < 0) rows_k = 0;
    if (c.split > 1) {  // part blockIdx.y of the rows, in whole slices
      const int n = cdiv(rows_k, P::kSK);
      const int a0 = (int)((int64_t)blockIdx.y * n / c.split), a1 = (int)((int64_t)(blockIdx.y + 1) * n / c.split);
      r0 += a0 * P::kSK;
      rows_k = min(rows_k - a0 * P::kSK, (a1 - a0) * P::kSK);
    }
    ex = __builtin_amdgcn_readfirstlane(ex);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    rows_k = __builtin_amdgcn_readfirstlane(rows_k);
  } else {
    int* s_off = reinterpret_cast<int*>(smem);
    load_tile_prefix<P::kBM, P::kFold>(c.offsets, c.e, c.A, s_off, s_off + 257);
    Tile t;
    if (!pick_tile<P::kBM, P::kBN, kGroup, P::kFold>(s_off, s_off + 257, c.e, MODE == GLU ? c.N : c.Hin, blockIdx.x, t))
      return;
    __syncthreads();  // every lane has its tile before the ring overwrites the prefix
    ex = t.ex;
    m0 = t.row0;
    mrows = t.rows;
    n0 = t.n0;
  }
  const int ncols = MODE == GLU ? c.N : MODE == DGRAD ? c.Hin : c.npair * c.N;
  const bool extra = P::kFold > 0 && mrows > P::kBM;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / P::kWavesN, wn = wave % P::kWavesN;
  const int ci = lane & 15, kq = lane >> 4;
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

  const int K = MODE == GLU ? c.Hin : MODE == DGRAD ? c.N : rows_k;
  const int nslice = cdiv(K, P::kSK);                       // of one operand pair
  const int nsteps = MODE == DGRAD ? c.npair * nslice : nslice;
  const uint32_t ldxb = (uint32_t)(MODE == DGRAD ? c.ldd : c.Hin) * (uint32_t)P::kES;
  const uint32_t ldwb = (uint32_t)(MODE == WGRAD ? c.ldd : c.ldw) * (uint32_t)P::kES;
  const bool gat = MODE != DGRAD && c.rm.src != nullptr;

  // ---- DMA sources: byte offsets of this lane for the KBs of a slot it fills
  // (two of x, one tail KB for waves 0 and 1, two of w); a set bit kOOB reads 0
  const unsigned char* xbase = reinterpret_cast<const unsigned char*>(MODE == DGRAD ? c.d[0] : c.x);
  u32x4_t xsrd, xsrd2, wsrd, wsrd2;
  uint32_t x_voff[3], x_kc[3], w_voff[2], w_kc[2];
  if (MODE == WGRAD) {
    if (gat) xsrd = make_srd(xbase, (uint32_t)c.rm.rows * ldxb);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int kb = (wave * 2 + q) * 1024 + lane * 16;
      const int k = kb / P::kXPitch;
      const uint32_t col = (uint32_t)P::source(P::kXPitch, k, kb % P::kXPitch);
      x_kc[q] = (uint32_t)(m0 * P::kES) + col;
      if (x_kc[q] >= (uint32_t)(c.Hin * P::kES)) x_kc[q] = kOOB;
      x_voff[q] = (uint32_t)k * ldxb + x_kc[q];
      w_kc[q] = (uint32_t)(n0 * P::kES) + col;
      if (w_kc[q] >= (uint32_t)(ncols * P::kES)) w_kc[q] = kOOB;
      w_voff[q] = (uint32_t)k * ldwb + w_kc[q];
    }
  } else {
    const int64_t xoff = gat ? 0 : (int64_t)m0 * ldxb;
    const uint32_t xbytes = (uint32_t)(gat ? c.rm.rows : mrows) * ldxb;
    xsrd = make_srd(xbase + xoff, xbytes);
    if (MODE == DGRAD && c.npair == 2)
      xsrd2 = make_srd(reinterpret_cast<const unsigned char*>(c.d[1]) + xoff, xbytes - (uint32_t)(c.N * P::kES));
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      if (q < 2 && q >= P::kXOps) continue;
      const int kb = (q < 2 ? (wave * P::kXOps + q) * 1024 : P::kBM * 64 + wave * 1024) + lane * 16;
      const int row = kb >> 6;
      x_kc[q] = (uint32_t)(((kb >> 4 & 3) ^ (row >> 1 & 3)) * 16);
      const int src = row >= mrows ? -1 : gat ? gather_src(c.rm, m0 + row) : row;
      x_voff[q] = (src >= 0 ? (uint32_t)src * ldxb : kOOB) + x_kc[q];
    }
    const int64_t wex = (int64_t)ex * c.Hin * c.ldw;
    const uint32_t wbytes = ((uint32_t)(c.Hin - 1) * (uint32_t)c.ldw + (uint32_t)c.N) * (uint32_t)P::kES;
    // GLU: the first half of the waves fills the gate panel, the others the up panel
    wsrd = make_srd(reinterpret_cast<const T*>(MODE == GLU && wm ? c.w[1] : c.w[0]) + wex, wbytes);
    if (MODE == DGRAD && c.npair == 2) wsrd2 = make_srd(reinterpret_cast<const T*>(c.w[1]) + wex, wbytes);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int kb = (wave * 2 + q) * 1024 + lane * 16;
      if (MODE == GLU) {
        const int pb = kb % (P::kLdsW / 2), k = pb / P::kWPitch;
        const uint32_t col = (uint32_t)(n0 * P::kES + P::source(P::kWPitch, k, pb % P::kWPitch));
        w_voff[q] = (uint32_t)k * ldwb + col;
        w_kc[q] = col < (uint32_t)(c.N * P::kES) ? 0u : kOOB;
      } else {
        const int row = kb >> 6;
        w_kc[q] = (uint32_t)(((kb >> 4 & 3) ^ (row >> 1 & 3)) * 16);
        w_voff[q] = (n0 + row < c.Hin ? (uint32_t)(n0 + row) * ldwb : kOOB) + w_kc[q];
      }
    }
  }
  // WGRAD gather: byte offsets of the source rows, 64 to a block: entry
  // kRW s + i is the wave's k row i of slice kSB b + s, and each of its two DMA
  // ops of a slice takes half of those rows. The index entries of block b+1 come by one DMA
  // op, three slices ahead of their first use, and are turned into offsets once
  // per block, one by each lane. (Any other load in the loop would be waited
  // for at the next barrier; entries fetched and divided for every slice took
  // 1460 us, these 1110 on 98304 rows of 2048 x 2816 over 64 experts, where
  // rows in order take 1080.) The op is not in the wait counts, which then
  // wait for one op more than they must in three slices of kSB.
  const uint32_t idx_lds = (uint32_t)P::kLds + wave * 512;
  u32x4_t isrd = {0u, 0u, 0u, 0u};
  if (MODE == WGRAD && gat) isrd = make_srd(c.rm.src + r0, (uint32_t)rows_k * 4u);
  auto k_entry = [&](int blk) { return (blk * P::kSB + lane / P::kRW) * P::kSK + wave * P::kRW + lane % P::kRW; };
  // Row v / div of x, or -1: the quotient by multiplication with
  // ceil(2^32 / div), which is exact or one too large for v < 2^31.
  const uint32_t div = (uint32_t)c.rm.div, recip = 0xffffffffu / div + 1u;
  auto offset_of = [&](int v, int k) {
    uint32_t q = div == 1u ? (uint32_t)v : __umulhi((uint32_t)v, recip);
    if (q * div > (uint32_t)v) --q;
    return k < rows_k && v >= 0 && q < (uint32_t)c.rm.rows ? q * ldxb : kOOB;
  };
  uint32_t* const idx_smem = reinterpret_cast<uint32_t*>(smem + idx_lds);
  if (MODE == WGRAD && gat) {
    const int k = k_entry(0);
    idx_smem[lane] = offset_of(k < rows_k ? c.rm.src[r0 + k] : 0, k);
  }
  uint32_t goff[2] = {0, 0};
  auto read_idx = [&](int step) {
    uint32_t* e = idx_smem + step / P::kSB % 2 * 64;
    if (step % P::kSB == 0 && step > 0) e[lane] = offset_of((int)e[lane], k_entry(step / P::kSB));
#pragma unroll
    for (int q = 0; q < 2; ++q) goff[q] = e[step % P::kSB * P::kRW + q * (P::kRW / 2) + lane / (128 / P::kRW)];
  };
  // Past-the-end slices are issued too (out-of-range loads write zeros), so
  // every wait count is fixed.
  // ex_: the tile carries tail rows; td: this wave fetches some of them (WGRAD: rows are gathered)
  auto issue = [&](int step, auto ex_, auto td) {
    const uint32_t base = lds0 + (step % S) * P::kStage;
    if (MODE == WGRAD) {
      const int k0 = step * P::kSK;
      const int left = rows_k - k0;  // k rows from here on
      const uint32_t n = left <= 0 ? 0u : left < P::kSK ? (uint32_t)left : (uint32_t)P::kSK;
      const int64_t row = r0 + (left > 0 ? k0 : 0);
      const u32x4_t ws = make_srd(reinterpret_cast<const unsigned char*>(c.d[0]) + row * ldwb, n * ldwb);
      if (decltype(td)::value) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t v = __builtin_elementwise_add_sat(goff[q], x_kc[q]);  // both may be out of range
          dma16(xsrd, v, base + (wave * 2 + q) * 1024);
        }
        const int next = step + S - 1;
        if (next % P::kSB == 0)
          dma4(isrd, (uint32_t)k_entry(next / P::kSB) * 4u, lds0 + idx_lds + next / P::kSB % 2 * 256);
      } else {
        const u32x4_t xs = make_srd(xbase + row * ldxb, n * ldxb);
#pragma unroll
        for (int q = 0; q < 2; ++q) dma16(xs, x_voff[q], base + (wave * 2 + q) * 1024);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) dma16(ws, w_voff[q], base + P::kLdsX + (wave * 2 + q) * 1024);
      return;
    }
    const bool second = MODE == DGRAD && step >= nslice && c.npair == 2;
    const int k0 = (second ? step - nslice : step) * 64;  // byte
    const u32x4_t xs = second ? xsrd2 : xsrd, ws = second ? wsrd2 : wsrd;
    const uint32_t kend = (uint32_t)(K * P::kES);
    const uint32_t past = step < nsteps ? 0u : kOOB;
#pragma unroll
    for (int q = 0; q < P::kXOps; ++q)
      dma16(xs, (x_voff[q] + k0) | (k0 + x_kc[q] < kend ? past : kOOB), base + (wave * P::kXOps + q) * 1024);
    if (decltype(ex_)::value && decltype(td)::value)
      dma16(xs, (x_voff[2] + k0) | (k0 + x_kc[2] < kend ? past : kOOB), base + P::kBM * 64 + wave * 1024);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t v = MODE == GLU ? (w_voff[q] + (uint32_t)(k0 / P::kES) * ldwb) | w_kc[q] | past
                                     : (w_voff[q] + k0) | (k0 + w_kc[q] < kend ? past : kOOB);
      dma16(ws, v, base + P::kLdsX + (wave * 2 + q) * 1024);
    }
  };

  // ---- fragments
  // of k rows: transposing reads, this lane naming 8 bytes of rows tr and tr + 4,
  // or (binary32) its column's four values from row tr on
  const int tr = kF32 ? 4 * kq : 8 * kq + (ci >> 2), trb = kF32 ? ci * 4 : (ci & 3) * 8;
  const int xsw = P::swz(P::kXPitch, tr), wsw = P::swz(P::kWPitch, tr);
  int xoff[P::kFI], xoff_t = 0, woff[4];
#pragma unroll
  for (int i = 0; i < P::kFI; ++i) {
    if (MODE == WGRAD) {
      xoff[i] = tr * P::kXPitch + ((wm * P::kFI + i) ^ xsw) * P::kUnit + trb;
    } else {
      const int m = (wm * P::kFI + i) * 16 + ci;
      xoff[i] = m * 64 + ((kq ^ (m >> 1 & 3)) << 4);
    }
  }
  if (P::kFold > 0) {
    const int m = P::kBM + wm * 16 + ci;
    xoff_t = m * 64 + ((kq ^ (m >> 1 & 3)) << 4);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (MODE == GLU) {
      woff[j] = (j >> 1) * (P::kLdsW / 2) + tr * P::kWPitch + ((wn * 2 + (j & 1)) ^ wsw) * P::kUnit + trb;
    } else if (MODE == WGRAD) {
      woff[j] = tr * P::kWPitch + ((wn * 4 + j) ^ wsw) * P::kUnit + trb;
    } else {
      const int n = wn * 64 + j * 16 + ci;
      woff[j] = n * 64 + ((kq ^ (n >> 1 & 3)) << 4);
    }
    woff[j] += P::kLdsX;
  }
  // 16 bytes of a row (column) per lane: k values 8 kq .. 8 kq + 7, or 4 kq .. 4 kq + 3
  typedef typename std::conditional<kF32, f32x4_t, bf16x8_t>::type Frag;
  auto read_tr = [&](const unsigned char* p, int pitch) {
    if constexpr (kF32) {
      f32x4_t v;
#pragma unroll
      for (int s = 0; s < 4; ++s) v[s] = *reinterpret_cast<const float*>(p + s * pitch);
      return v;
    } else {
      typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;
      const i16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
      const i16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 4 * pitch));
      typedef short i16x8_t __attribute__((ext_vector_type(8)));
      return __builtin_bit_cast(bf16x8_t, (i16x8_t)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };
  struct Frags {
    Frag x[P::kFI], t, w[4];
  };
  auto read_frags = [&](int slice, Frags& f, auto ex_) {
    const unsigned char* st = smem + (slice % S) * P::kStage;
#pragma unroll
    for (int i = 0; i < P::kFI; ++i)
      f.x[i] = MODE == WGRAD ? read_tr(st + xoff[i], P::kXPitch) : *reinterpret_cast<const Frag*>(st + xoff[i]);
    if (decltype(ex_)::value) f.t = *reinterpret_cast<const Frag*>(st + xoff_t);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f.w[j] = MODE == DGRAD ? *reinterpret_cast<const Frag*>(st + woff[j]) : read_tr(st + woff[j], P::kWPitch);
  };
  f32x4_t acc[P::kFI][4], acct[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int i = 0; i < P::kFI; ++i) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    acct[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  }
  auto multiply = [&](const Frags& f, auto ex_) {
    if constexpr (kF32) {  // MFMA s takes k values 4 kq + s
#pragma unroll
      for (int i = 0; i < P::kFI; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(f.w[j][s], f.x[i][s], acc[i][j], 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < P::kFI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.w[j], f.x[i], acc[i][j], 0, 0, 0);
      if (decltype(ex_)::value) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acct[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.w[j], f.t, acct[j], 0, 0, 0);
      }
    }
  };
  // binary32: the sums of 128 k values at a time are added to totals, which keeps
  // the rounding from growing with the reduction (one running sum over 4096
  // normal products is off by 1.1e-6 of the result's norm, this by 2.3e-7)
  f32x4_t tot[kF32 ? P::kFI : 1][kF32 ? 4 : 1];
  auto to_totals = [&](bool first) {
    if constexpr (kF32) {
#pragma unroll
      for (int i = 0; i < P::kFI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tot[i][j] = first ? acc[i][j] : tot[i][j] + acc[i][j];
          acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        }
    }
  };
  to_totals(true);
  const int wcols = MODE == GLU ? 32 : 64;  // output columns per wave
  const bool active = wm * (P::kBM / 2) < mrows && n0 + wn * wcols < ncols;
  // Element (row, col) of a weight gradient's tile: dg's or du's, of this part.
  auto wgrad_at = [&](int row, int col) {
    const bool second = col >= c.N;  // N is a multiple of 8 (binary32: 4): 16 bytes have one owner
    const int64_t part = (int64_t)blockIdx.y * c.e * c.Hin * c.ldw;  // of the partial sums
    return reinterpret_cast<TO*>(second ? c.out[1] : c.out[0]) + part +
           ((int64_t)ex * c.Hin + m0 + row) * c.ldw + (second ? col - c.N : col);
  };
  // binary32 results of bf16 operands: an expert may have any number of rows, and
  // totals would not fit beside the large tiles' accumulators, so the sums of 4096
  // rows at a time are added to the output, by the lane that wrote those before.
  // (One sum over 65536 normal products is off by 1.6e-6 of the result's norm, over
  // 262144 by 3.3e-6, these by 4.0e-7 and 4.2e-7. 98304 rows of 2048 x 2816, 64
  // experts, the longest of 28865 rows: 1162 us without, 1234 so; experts of up to
  // 4096 rows as before.) bf16 results, rounded to 2^-9, do without.
  constexpr bool kPieces = MODE == WGRAD && sizeof(TO) == 4 && !kF32;
  constexpr int kPiece = 4096 / P::kSK;  // slices
  const bool pieces = kPieces && c.pieces;
  bool held = false;  // the output holds this wave's sums of earlier rows
  auto add_piece = [&]() __attribute__((always_inline)) {
    if constexpr (kPieces) {
      // opaque, so that no address is held in registers through the loop
      int row = wm * P::kFI * 16 + ci, col = n0 + wn * 64 + 4 * kq;
      asm volatile("" : "+v"(row), "+v"(col));
#pragma unroll
      for (int i = 0; i < P::kFI; ++i) {
        if (active && row < mrows) {
          // a row's earlier sums together, so that their loads overlap
          f32x4_t v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
            if (held && col + j * 16 < ncols) v[j] = *reinterpret_cast<const f32x4_t*>(wgrad_at(row, col + j * 16));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col + j * 16 < ncols) *reinterpret_cast<f32x4_t*>(wgrad_at(row, col + j * 16)) = v[j] + acc[i][j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        row += 16;
        asm volatile("" : "+v"(row));
        __builtin_amdgcn_sched_barrier(0);
      }
      held = true;
    }
  };
  // The compiler may not move work across these barriers: the phases are the schedule.
  auto bar = [] {
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto run = [&](auto ex_, auto td) {
    constexpr bool kGat = MODE == WGRAD && decltype(td)::value;
    constexpr int kInFlight = (S - 2) * (P::kXOps + 2 + (decltype(ex_)::value && decltype(td)::value ? 1 : 0));
    // before the fragments, so that the offsets' wait leaves those reads in flight
    auto ahead = [&](int step) {
      if (kGat) read_idx(step);
    };
    auto put = [&](int step) { issue(step, ex_, td); };
#pragma unroll
    for (int t = 0; t < S - 1; ++t) {
      ahead(t);
      put(t);
    }
    wait_vmcnt<kInFlight>();
    bar();  // barrier 0: slice 0 has landed
    Frags f;
    if constexpr (SIZE != LARGE) {
      Frags g;
      ahead(S - 1);
      read_frags(0, f, ex_);
      put(S - 1);
      auto step = [&](int s, const Frags& now, Frags& next) {
        wait_vmcnt<kInFlight>();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        bar();  // slice s+1 has landed; every wave holds its fragments of slice s
        ahead(s + S);
        read_frags(s + 1, next, ex_);
        put(s + S);
        if (!kF32 || active) multiply(now, ex_);
      };
      for (int s = 0; s < nsteps; s += 2) {
        step(s, f, g);
        if (s + 1 < nsteps) step(s + 1, g, f);
        if (kF32 && (s + 2) * P::kSK % 128 == 0) to_totals(false);
        if (pieces && (s + 2) % kPiece == 0 && s + 2 < nsteps) add_piece();
      }
      if constexpr (kF32) {
        to_totals(false);
#pragma unroll
        for (int i = 0; i < P::kFI; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = tot[i][j];
      }
      return;
    }
    if (wm == 0) {
      if (active) {
        ahead(S - 1);
        read_frags(0, f, ex_);
        put(S - 1);
        bar();
        for (int s = 0; s < nsteps; ++s) {
          multiply(f, ex_);
          if (pieces && (s + 1) % kPiece == 0 && s + 1 < nsteps) add_piece();
          wait_vmcnt<kInFlight>();
          bar();
          ahead(s + S);
          read_frags(s + 1, f, ex_);
          put(s + S);
          bar();
        }
      } else {
        ahead(S - 1);
        put(S - 1);
        bar();
        for (int s = 0; s < nsteps; ++s) {
          wait_vmcnt<kInFlight>();
          bar();
          ahead(s + S);
          put(s + S);
          bar();
        }
      }
      bar();  // matches the second half's last barrier
    } else {
      bar();
      ahead(S - 1);
      put(S - 1);
      if (active) {
        read_frags(0, f, ex_);
        wait_vmcnt<kInFlight>();
        bar();
        for (int s = 0; s < nsteps; ++s) {
          multiply(f, ex_);
          if (pieces && (s + 1) % kPiece == 0 && s + 1 < nsteps) add_piece();
          bar();
          ahead(s + S);
          read_frags(s + 1, f, ex_);
          put(s + S);
          wait_vmcnt<kInFlight>();
          bar();
        }
      } else {
        wait_vmcnt<kInFlight>();
        bar();
        for (int s = 0; s < nsteps; ++s) {
          bar();
          ahead(s + S);
          put(s + S);
          wait_vmcnt<kInFlight>();
          bar();
        }
      }
    }
  };
  if constexpr (P::kFold == 0) {
    if (gat) run(std::false_type{}, std::true_type{});
    else run(std::false_type{}, std::false_type{});
  } else {
    if (!extra) run(std::false_type{}, std::false_type{});
    else if (wave < 2) run(std::true_type{}, std::true_type{});
    else run(std::true_type{}, std::false_type{});
  }
  wait_vmcnt<0>();  // no DMA may still be landing when the block's LDS is reused
  if (pieces && nsteps > kPiece) {  // for every wave, with or without sums of its own
    add_piece();
    return;
  }
  __syncthreads();

  // ---- epilogue: fragment i's row (kFI: the tail), columns 4 kq .. 4 kq + 3 of n fragment j
  auto frag_row = [&](int i) { return i < P::kFI ? (wm * P::kFI + i) * 16 + ci : P::kBM + wm * 16 + ci; };
  constexpr int kFrags = P::kFI + (P::kFold > 0 ? 1 : 0);
  // Copies nrows staged rows (tile rows from `first` on) to rows of `o`.
  auto copy_rows = [&](int first, int nrows, auto dst) {
    constexpr int kPer = 16 / (int)sizeof(TO);          // columns per 16 bytes
    constexpr int kLanes = P::kBN / kPer;               // lanes per row
#pragma unroll 1
    for (int idx = tid; idx < nrows * kLanes; idx += P::kNT) {
      const int row = idx / kLanes, col = idx % kLanes * kPer;
      if (n0 + col >= ncols) continue;
      *reinterpret_cast<uint4*>(dst(first + row, n0 + col)) =
          *reinterpret_cast<const uint4*>(smem + row * P::kOutRow + col * (int)sizeof(TO));
    }
  };
  if constexpr (MODE == GLU) {
    // OUT: 0 act(g) * u with activation ACT, 1 g, 2 u
    auto stage = [&](auto OUT, auto ACT) {
      constexpr int kOut = decltype(OUT)::value;
      if (!active) return;
#pragma unroll
      for (int i = 0; i < kFrags; ++i) {
        if (i == P::kFI && !extra) continue;  // compile-time i keeps the accumulators in registers
        const int ml = frag_row(i);
        if (ml >= mrows) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const f32x4_t g = i < P::kFI ? acc[i][j] : acct[j], u = i < P::kFI ? acc[i][j + 2] : acct[j + 2];
          float v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            v[r] = kOut == 0 ? act_of<!kF32>(g[r], decltype(ACT)::value) * u[r] : kOut == 1 ? g[r] : u[r];
          unsigned char* o = smem + ml * P::kOutRow + (wn * 32 + j * 16 + 4 * kq) * P::kES;
          if (kF32)
            *reinterpret_cast<f32x4_t*>(o) = (f32x4_t){v[0], v[1], v[2], v[3]};
          else
            *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        }
      }
    };
    auto store = [&](void* o) {
      __syncthreads();
      T* out = reinterpret_cast<T*>(o);
      copy_rows(0, mrows, [&](int row, int col) { return out + (int64_t)(m0 + row) * c.N + col; });
    };
    typedef std::integral_constant<int, 0> I0;
    typedef std::integral_constant<int, 1> I1;
    typedef std::integral_constant<int, 2> I2;
    if (c.act == MOE_ACT_SILU) stage(I0{}, std::integral_constant<int, MOE_ACT_SILU>{});
    else if (c.act == MOE_ACT_GELU) stage(I0{}, std::integral_constant<int, MOE_ACT_GELU>{});
    else if (c.act == MOE_ACT_RELU) stage(I0{}, std::integral_constant<int, MOE_ACT_RELU>{});
    else stage(I0{}, std::integral_constant<int, MOE_ACT_NONE>{});
    store(c.out[0]);
    if (c.out[1] != nullptr) {
      __syncthreads();
      stage(I1{}, I0{});
      store(c.out[1]);
      __syncthreads();
      stage(I2{}, I0{});
      store(c.out[2]);
    }
  } else {
#pragma unroll
    for (int ps = 0; ps < P::kPasses; ++ps) {
      const int first = ps * 128;
      if (ps > 0) __syncthreads();
      if (active && (P::kPasses == 1 || wm == ps)) {
#pragma unroll
        for (int i = 0; i < kFrags; ++i) {
          if (i == P::kFI && !extra) continue;
          const int ml = frag_row(i);
          if (ml >= mrows) continue;
          unsigned char* lrow = smem + (ml - first) * P::kOutRow;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4_t v = i < P::kFI ? acc[i][j] : acct[j];
            const int col = wn * 64 + j * 16 + 4 * kq;
            if (sizeof(TO) == 4)
              *reinterpret_cast<f32x4_t*>(lrow + col * 4) = v;
            else
              *reinterpret_cast<uint2*>(lrow + col * 2) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
          }
        }
      }
      __syncthreads();
      const int left = mrows - first;
      const int nrows = P::kPasses == 1 ? left : left < 0 ? 0 : left < 128 ? left : 128;
      copy_rows(first, nrows, [&](int row, int col) {
        if (MODE == DGRAD) return reinterpret_cast<TO*>(c.out[0]) + (int64_t)(m0 + row) * c.Hin + col;
        return wgrad_at(row, col);
      });
    }
  }
}

// Largest dynamic LDS allowed for a kernel, set once per device.
template <typename Kern>
void allow_lds(Kern* k, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  const uint64_t bit = 1ull << dev;
  if (done.load(std::memory_order_relaxed) & bit) return;
  (void)hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  done.fetch_or(bit, std::memory_order_relaxed);
}

// Sum of the partial weight gradients in part order, 8 columns per lane:
// part (split, e, Hin, np * N) -> out[p] (e, Hin, N of ld).
template <typename TO>
__global__ __launch_bounds__(256) void sum_parts_kernel(const float* __restrict__ part, FfnCall c, TO* out0, TO* out1,
                                                        int64_t rows) {
  const int cols = c.npair * c.N, per = cols / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / per;
  if (row >= rows) return;
  const int col = (int)(i - row * per) * 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int q = 0; q < c.split; ++q) {
    const float4* p = reinterpret_cast<const float4*>(part + ((int64_t)q * rows + row) * cols + col);
    const float4 a = p[0], b = p[1];
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
  }
  TO* o = (col >= c.N ? out1 : out0) + row * c.ldw + (col >= c.N ? col - c.N : col);
  if constexpr (sizeof(TO) == 4) {
    reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

template <int MODE>
double tile_count(const FfnCall& c, int bm) {
  const int ncols = MODE == GLU ? c.N : MODE == DGRAD ? c.Hin : c.npair * c.N, bn = bm == 64 ? 128 : bm;
  const double cols = cdiv(ncols, MODE == GLU ? bn / 2 : bn);
  if (MODE == WGRAD) return (double)c.e * cdiv(c.Hin, bm) * cols;
  const double experts = c.e < c.A ? c.e : c.A;
  return (experts == 1 ? (double)cdiv(c.A, bm) : (double)c.A / bm + experts / 2) * cols;
}
// Estimated time of a launch in microseconds, from what the two tile sizes
// measured over 16 shapes of 64 to 16384 rows: per 32-deep slice and per tile
// outside its loop, with one tile per CU (large) or two (small; a CU left with
// one small tile runs it faster). Rows per expert are taken as the average,
// with half a tile of slack for each expert; the estimates only choose between
// sizes and splits, which give the same sums up to the order of additions.
// Examples, measured (large / small): GLU of 512 rows, 4096 -> 4096, one expert
// 78 / 42 us; 4503 rows, 744 -> 1056, 16 experts 28 / 35; weight gradients of
// 8192 rows, 1024 x 768, 64 experts 52 / 44; 8192 rows, 4096 x 14336, 8
// experts 967 / 1100.
template <int MODE>
double tiles_time(const FfnCall& c, bool small, int split, int ncu) {
  const int bm = small ? 128 : 256;
  const bool f32 = c.dt == MOE_F32;
  const int sk = f32 ? 16 : 32;
  const double tiles = tile_count<MODE>(c, bm) * split;
  const double slices = MODE == WGRAD ? (double)c.A / c.e / sk / split : MODE == GLU ? cdiv(c.Hin, sk)
                                                                                     : c.npair * cdiv(c.N, sk);
  const double per = small ? 2.0 * ncu : ncu;
  const double full = (double)(int64_t)(tiles / per), rest = tiles - full * per;
  if (f32) return full * (1.8 * slices + 7) + (rest > ncu ? 1.8 * slices + 7 : rest > 0 ? 1.0 * slices + 7 : 0);
  if (!small) return (full + (rest > 0)) * ((MODE == WGRAD ? 0.66 : 0.70) * slices + 15);
  const double two = MODE == WGRAD ? 0.42 * slices + 7 : 0.60 * slices + 6;
  const double one = MODE == WGRAD ? 0.25 * slices + 7 : 0.30 * slices + 6;
  return full * two + (rest > ncu ? two : rest > 0 ? one : 0);
}
// binary32: 64 x 128 tiles, three per CU, which lose less to ragged experts and
// to the last round; 128 x 128 for one expert with many tiles. (128 x 128 / 64 x
// 128, us: GLU of 16384 rows, 1000 -> 1100, 64 experts 781 / 694; 2048 rows, 4096
// -> 2048, 8 experts 788 / 664; dgrad of 8192 rows, 2048 -> 1024, one expert 270 /
// 289.)
template <int MODE>
bool f32_flat(const FfnCall& c, int ncu) {
  return c.e > 1 || tile_count<MODE>(c, 128) < 2.0 * ncu;
}
template <int MODE>
bool takes_small(const FfnCall& c, int split, int ncu) {
  return tiles_time<MODE>(c, true, split, ncu) < tiles_time<MODE>(c, false, split, ncu);
}

// Parts the rows of every expert are split into for the weight gradients: with
// few output tiles (a dense FFN, a few small experts) most CUs would have none.
// Writing and reading back the binary32 partial sums takes 0.11 us per part and
// 256 x 256 elements. (98304 rows of 2048 x 2816, one expert: 2113 us whole,
// 1053 in 8 parts.)
int wgrad_split(const FfnCall& c, int ncu) {
  const double elems = (double)c.e * c.Hin * c.npair * c.N / 65536;
  int best = 1;
  double least = 0;
  if (c.N % 8 != 0) return 1;  // sum_parts_kernel's eight columns have one owner
  for (int S = 1; S <= 16; ++S) {
    if (S > 1 && (S * elems > 8.0 * ncu || (int64_t)S * c.e * 256 > c.A)) break;
    const double l = tiles_time<WGRAD>(c, false, S, ncu), t = tiles_time<WGRAD>(c, true, S, ncu);
    const double cost = (l < t ? l : t) + (S > 1 ? 0.11 * S * elems + 5 : 0);
    if (S == 1 || cost < least) {
      least = cost;
      best = S;
    }
  }
  return best;
}

template <int MODE, typename TO, int SIZE, typename T>
moe_status launch_size(const FfnCall& c, hipStream_t s) {
  typedef PpTile<MODE, TO, SIZE, T> P;
  static std::atomic<uint64_t> done{0};
  allow_lds(&ffn_pp_kernel<MODE, TO, SIZE, T>, P::kLds + P::kIdx, done);
  const int ncols = MODE == GLU ? c.N : MODE == DGRAD ? c.Hin : c.npair * c.N;
  int64_t grid;
  if (MODE == WGRAD)
    grid = (int64_t)c.e * 8 * cdiv(cdiv(c.Hin, P::kBM) * cdiv(ncols, P::kBN), 8);
  else
    grid = cdiv64((cdiv64(c.A, P::kBM) + (c.e < c.A ? c.e : c.A)) * cdiv(ncols, P::kBN), 8) * 8;
  if (grid > 0x7fffffff) return MOE_ERR_BAD_SHAPE;
  hipLaunchKernelGGL((ffn_pp_kernel<MODE, TO, SIZE, T>), dim3((unsigned)grid, MODE == WGRAD ? c.split : 1), dim3(P::kNT),
                     P::kLds + P::kIdx, s, c);
  return launch_status();
}

template <int MODE, typename TO>
moe_status launch_mode(const FfnCall& c, hipStream_t s) {
  if constexpr (sizeof(TO) == 4) {
    if constexpr (MODE != WGRAD) {
      if (c.dt == MOE_F32 && f32_flat<MODE>(c, device_cus())) return launch_size<MODE, TO, FLAT, float>(c, s);
    }
    if (c.dt == MOE_F32) return launch_size<MODE, TO, SMALL, float>(c, s);
  }
  if constexpr (sizeof(TO) == 2 || MODE == WGRAD) {
    return takes_small<MODE>(c, c.split, device_cus()) ? launch_size<MODE, TO, SMALL, bf16_t>(c, s)
                                                       : launch_size<MODE, TO, LARGE, bf16_t>(c, s);
  }
  return MOE_ERR_BAD_DTYPE;  // not reached
}

}  // namespace

namespace {
// Every row on 16 bytes, an expert's weights within 31-bit byte offsets.
bool aligned(const FfnCall& c) {
  const int es = c.dt == MOE_F32 ? 4 : 2, q = 16 / es;
  return c.Hin % q == 0 && c.N % q == 0 && c.ldw % q == 0 && (int64_t)c.Hin * c.ldw * es < (1ll << 31);
}
}  // namespace

// binary32 has the 32 x 64 tiles of ffn_tile_kernel for calls with few tiles (64 x
// 128 / 32 x 64, us: GLU of 256 rows, 1024 -> 1024, 16 experts, 192 tiles, 45 / 61;
// 1000 rows, 512 -> 512, 4 experts, 141 tiles, 25 / 29; 128 rows, 2048 -> 2048,
// 64 tiles, 81 / 41; dgrad of 2048 rows, 1024 -> 1024, 4 experts, 272 tiles, 77 /
// 59; 4096 rows, 2048 -> 2048, 4 experts, 1056 tiles, 352 / 454).
bool glu_pp_takes(const FfnCall& c) {
  return aligned(c) && (c.dt == MOE_BF16 || 2 * tile_count<GLU>(c, 64) >= device_cus());
}
bool dgrad_pp_takes(const FfnCall& c) {
  return aligned(c) && (c.dt == MOE_BF16 || tile_count<DGRAD>(c, 64) >= 2 * device_cus());
}
// ... and weight gradients with few tiles and few rows to split (9001 rows, 264 x
// 136, one expert, 6 tiles in 16 parts, 53 / 174; 4096 rows, 128 x 64, 2 experts
// 28 / 43; 4096 rows, 512 x 128, 4 experts 28 / 25).
bool wgrad_pp_takes(const FfnCall& c) {
  if (!aligned(c) || c.dt == MOE_BF16) return aligned(c);
  const int S = wgrad_split(c, device_cus());
  return (S >= 4 && c.A >= 2048ll * c.e) || 4 * tile_count<WGRAD>(c, 128) * S >= 3 * device_cus();
}
moe_status launch_glu_pp(const FfnCall& c, hipStream_t s) {
  return c.dt == MOE_F32 ? launch_mode<GLU, float>(c, s) : launch_mode<GLU, bf16_t>(c, s);
}
moe_status launch_dgrad_pp(const FfnCall& c, hipStream_t s) {
  return c.dt == MOE_F32 ? launch_mode<DGRAD, float>(c, s) : launch_mode<DGRAD, bf16_t>(c, s);
}
size_t wgrad_pp_ws(const FfnCall& c) {
  const int S = wgrad_split(c, device_cus());
  return S > 1 ? (size_t)S * c.e * c.Hin * c.npair * c.N * sizeof(float) : 0;
}
moe_status launch_wgrad_pp(const FfnCall& c0, moe_dtype out_dt, void* ws, hipStream_t s) {
  FfnCall c = c0;
  c.split = wgrad_split(c, device_cus());
  c.pieces = out_dt == MOE_F32;
  if (c.split == 1) return out_dt == MOE_F32 ? launch_mode<WGRAD, float>(c, s) : launch_mode<WGRAD, bf16_t>(c, s);
  FfnCall p = c;
  p.ldw = c.npair * c.N;
  p.out[0] = ws;
  p.out[1] = (float*)ws + c.N;
  const moe_status st = launch_mode<WGRAD, float>(p, s);
  if (st != MOE_OK) return st;
  const int64_t rows = (int64_t)c.e * c.Hin;
  const int64_t grid = cdiv64(rows * (p.ldw / 8), 256);
  if (grid > 0x7fffffff) return MOE_ERR_BAD_SHAPE;
  if (out_dt == MOE_F32)
    hipLaunchKernelGGL(sum_parts_kernel<float>, dim3((unsigned)grid), dim3(256), 0, s, (const float*)ws, c,
                       (float*)c.out[0], (float*)c.out[1], rows);
  else
    hipLaunchKernelGGL(sum_parts_kernel<bf16_t>, dim3((unsigned)grid), dim3(256), 0, s, (const float*)ws, c,
                       (bf16_t*)c.out[0], (bf16_t*)c.out[1], rows);
  return launch_status();
}

}  // namespace moe
