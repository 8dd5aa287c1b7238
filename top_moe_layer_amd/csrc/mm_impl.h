// Products of grouped rows on the matrix cores (gfx950, wave64): the tile
// kernel.  Layouts and formats: mm.h.
//
// A block of WM x WN wavefronts computes a BM x BN tile of C.  K advances in
// slices of KS elements, fetched straight into a ring of S LDS slots
// (buffer_load ... lds, 16 bytes a lane); a wavefront holds its piece of C in
// 32 x 32 accumulators and double-buffers the fragments of a slice's sub-steps
// in registers.  Loads go through buffer descriptors that end with the tile's
// last row, and lanes past the last column or past K load from beyond them:
// such loads deliver zeros, so ragged groups, odd sizes and K tails need no
// code in the loop, and a zero meets a zero (or a valid scale) everywhere.
//
// LDS layouts.  An operand whose rows run along K keeps KS elements a row, its
// 16-byte chunks at chunk ^ ((row * RB / 256) % chunks): fragment reads are
// free of bank conflicts.  One whose rows run across K (the matrix of NN, both
// operands of TN) is kept as it lies in memory, KS rows of BX columns; bf16
// fragments come out of it through the transposing LDS read
// (ds_read_b64_tr_b16: of 16 lanes that read four rows of 16 columns each ends
// with the four values of a column), rows k, k + 1, k + 2, k + 3 sitting in
// different 64-byte units by unit ^ (k % 4).  So neither dx nor dw transposes
// anything in memory.
//
// Matrix instructions, all with fp32 accumulators:
//   bf16           32x32x16 (a lane holds 8 k)
//   fp32           32x32x2, four for a lane's 4 k
//   fp32 rows beside bf16 or e2m1 matrices: x = hi + mid + lo, three bf16 parts
//                  by truncation, exact; three bf16 instructions instead of
//                  eight fp32 ones at a sixteenth of the rate
//   e2m1 matrix beside bf16 rows: 16 bytes of a lane are its 32 k of a slice,
//                  turned into bf16 with their scale (exact) as they are used
//   e2m1 x e2m1, e4m3 x e2m1: 32x32x64 with the scales as operands
#pragma once

#include <type_traits>

#include "device_common.h"
#include "mm.h"

namespace topmoe {
namespace mm {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// (Out of the kernel templates, where a target builtin would suppress the host stub.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), short(0), int(bytes), 0x00020000);
}
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16,
                                           int(off), 0, 0, 0);
}
__device__ __forceinline__ u32x2 read_tr(const char* lds) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4*)lds));
}
__device__ __forceinline__ const char* scalar_ptr(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  return reinterpret_cast<const char*>((uint64_t(hi) << 32) | lo);
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
// Every wavefront's own loads have landed (the caller waited) and its LDS reads
// are done: the slot read so far may be refilled, the next one read.
__device__ __forceinline__ void slot_barrier() {
  __builtin_amdgcn_s_waitcnt((7 << 4) | (0 << 8) | 0xC00F);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}
constexpr uint32_t kBeyond = 0x80000000u;  // an offset past every buffer

__device__ __forceinline__ f32x16 mfma_bf16(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma_f32(u32x4 a, u32x4 b, f32x16 c) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[s]), __uint_as_float(b[s]), c, 0, 0,
                                             0);
  return c;
}
// FA: 0 e4m3 (eight registers), 4 e2m1 (four); byte SEL of the scales.
template <int FA, int SEL>
__device__ __forceinline__ f32x16 mfma_mx(u32x4 a0, u32x4 a1, u32x4 b, f32x16 c, uint32_t sa,
                                          uint32_t sb) {
  const i32x8 x = {int(a0[0]), int(a0[1]), int(a0[2]), int(a0[3]),
                   int(a1[0]), int(a1[1]), int(a1[2]), int(a1[3])};
  const i32x8 y = {int(b[0]), int(b[1]), int(b[2]), int(b[3]), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, FA, 4, SEL, int(sa), SEL,
                                                         int(sb));
}
// Two e2m1 / e4m3 values times a scale as two bf16 (exact; a product outside
// bf16's range becomes infinite, or rounds on its subnormals).
template <int SEL>
__device__ __forceinline__ uint32_t bf16_of_e2m1(uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, SEL));
}
template <bool HIGH>
__device__ __forceinline__ uint32_t bf16_of_e4m3(uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, HIGH));
}
__device__ __forceinline__ u32x4 bf16_of_e2m1x8(uint32_t w, float s) {
  return u32x4{bf16_of_e2m1<0>(w, s), bf16_of_e2m1<1>(w, s), bf16_of_e2m1<2>(w, s),
               bf16_of_e2m1<3>(w, s)};
}
__device__ __forceinline__ u32x4 bf16_of_e4m3x8(uint32_t w0, uint32_t w1, float s) {
  return u32x4{bf16_of_e4m3<false>(w0, s), bf16_of_e4m3<true>(w0, s), bf16_of_e4m3<false>(w1, s),
               bf16_of_e4m3<true>(w1, s)};
}
// Eight fp32 values (of two 16-byte pieces) as three bf16 parts whose sum they
// are: the upper 8 bits of the mantissa, of the rest and of its rest, 24 in all.
// An infinity is its own first part, with no rest; NaN leaves NaN in the rest.
__device__ __forceinline__ void split3(u32x4 a, u32x4 b, u32x4 (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[2], m[2], l[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float x = __uint_as_float(i < 2 ? a[2 * i + t] : b[2 * i - 4 + t]);
      const float hi = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
      const float r = x == hi ? 0.f : x - hi;
      h[t] = __float_as_uint(hi);
      m[t] = __float_as_uint(r) & 0xffff0000u;
      l[t] = __float_as_uint(r - __uint_as_float(m[t]));
    }
    p[0][i] = (h[0] >> 16) | h[1];
    p[1][i] = (m[0] >> 16) | m[1];
    p[2][i] = (l[0] >> 16) | (l[1] & 0xffff0000u);
  }
}
// 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float scale_f32(uint32_t byte) {
  return byte == 0 ? __uint_as_float(0x00400000u)
                   : byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// n scale bytes (1, 2 or 4) from kb on of a row of KB, 2^0 behind its end.
template <int n>
__device__ __forceinline__ uint32_t scale_bytes(const uint8_t* row, int kb, int KB) {
  if (kb + n <= KB) {
    if constexpr (n == 4) {
      typedef uint32_t __attribute__((aligned(1))) w;
      return *reinterpret_cast<const w*>(row + kb);
    } else if constexpr (n == 2) {
      typedef uint16_t __attribute__((aligned(1))) w;
      return *reinterpret_cast<const w*>(row + kb);
    } else {
      return row[kb];
    }
  }
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) v |= uint32_t(kb + i < KB ? row[kb + i] : 127) << (8 * i);
  return v;
}

// The offsets' expert e, held inside [0, R] so that no row outside is touched
// whatever the array holds; expert 0 starts at row 0.
__device__ __forceinline__ int offset_at(const int32_t* offsets, int e, int E, int64_t R) {
  if (e <= 0) return 0;
  const int o = offsets[e < E ? e : E];
  return o < 0 ? 0 : o > R ? int(R) : o;
}

// The group of row tile t, with its first row and the rows from there on; the
// tiles behind the experts' hold the rows of no expert (e == E).  Each
// wavefront finds it by itself, a lane holding four experts.
struct RowTile {
  int e, row0, rows;
};
template <int BM>
__device__ __forceinline__ int row_tiles(const int32_t* offsets, int E, int64_t R, int lane,
                                         int (&o)[5], int& incl, int& last) {
#pragma unroll
  for (int i = 0; i < 5; ++i) o[i] = offset_at(offsets, 4 * lane + i, E, R);
  int mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = o[i + 1] - o[i];
    if (4 * lane + i < E && c > 0) mine += (c + BM - 1) / BM;
  }
  incl = wave_inclusive_scan(mine, lane);
  last = offset_at(offsets, E, E, R);
  const int real = __builtin_amdgcn_readlane(incl, 63);
  return real + int((R - last + BM - 1) / BM);
}
template <int BM>
__device__ __forceinline__ RowTile row_tile(int t, const int (&o)[5], int incl, int last, int E,
                                            int64_t R, int lane) {
  const uint64_t before = __ballot(incl <= t);
  const int at = __popcll(before);  // lanes whose tiles all precede t
  RowTile r;
  if (at >= 64) {
    r.e = E;
    r.row0 = last + (t - __builtin_amdgcn_readlane(incl, 63)) * BM;
    r.rows = int(R) - r.row0;
  } else {
    int left = t - (at > 0 ? __builtin_amdgcn_readlane(incl, at - 1) : 0);
    r.e = 4 * at;
    r.row0 = r.rows = 0;
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = __builtin_amdgcn_readlane(o[i], at), b = __builtin_amdgcn_readlane(o[i + 1], at);
      const int tiles = b > a ? (b - a + BM - 1) / BM : 0;
      if (!found && left < tiles) {
        found = true;
        r.e = 4 * at + i;
        r.row0 = a + left * BM;
        r.rows = b - r.row0;
      }
      left -= tiles;
    }
  }
  r.rows = r.rows < BM ? r.rows : BM;
  return r;
}

// Elements of a K slice.
constexpr int slice_of(int fa, int fb) {
  return fa == kMmF32 ? 32 : fb == kMmE2m1 ? (fa == kMmE2m1 ? 256 : 128) : 64;
}

template <int LAYOUT, int FA, int FB, typename OT, int BM, int BN, int WM, int WN, int S>
struct Shape {
  static constexpr int KS = slice_of(FA, FB);
  static constexpr bool TA = LAYOUT == kMmTN, TB = LAYOUT != kMmNT;  // rows across K
  static constexpr int RBA = TA ? BM * mm_bits(FA) / 8 : KS * mm_bits(FA) / 8;  // bytes of an LDS row
  static constexpr int RBB = TB ? BN * mm_bits(FB) / 8 : KS * mm_bits(FB) / 8;
  static constexpr int ABYTES = BM * KS * mm_bits(FA) / 8, BBYTES = BN * KS * mm_bits(FB) / 8;
  static constexpr int STAGE = ABYTES + BBYTES;
  static constexpr int NW = WM * WN;
  static constexpr int LA = (ABYTES / 1024 + NW - 1) / NW, LB = (BBYTES / 1024 + NW - 1) / NW;
  // two blocks a CU where their rings fit, else one
  static constexpr int WAVES = (2 * S * STAGE <= 160 * 1024 ? 2 : 1) * (NW > 4 ? NW / 4 : 1);  // a SIMD
  static constexpr int LMIN = ABYTES / 1024 / NW + BBYTES / 1024 / NW;  // fewest loads of a wavefront
};

// Chunk position of row `row` in rows of RB bytes along K.
template <int RB>
__device__ __forceinline__ int swz(int row) {
  return (row * RB / 256) % (RB / 16);
}
// The same for rows across K: 16-byte chunks move by whole 64-byte units (bf16)
// or 128-byte halves (fp32, where lanes 0-31 and 32-63 read rows k and k + 4).
template <int BITS>
__device__ __forceinline__ int swz_t(int row) {
  return BITS == 16 ? (row & 3) * 4 : ((row >> 2) & 1) * 8;
}

template <int LAYOUT, int FA, int FB, typename OT, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN, (Shape<LAYOUT, FA, FB, OT, BM, BN, WM, WN, S>::WAVES))
void mm_kernel(MmParams p) {
  using Z = Shape<LAYOUT, FA, FB, OT, BM, BN, WM, WN, S>;
  constexpr int KS = Z::KS, NW = Z::NW, RBA = Z::RBA, RBB = Z::RBB, STAGE = Z::STAGE;
  constexpr bool TA = Z::TA, TB = Z::TB, TN_ = LAYOUT == kMmTN;
  constexpr bool MX = FB == kMmE2m1, F32 = FA == kMmF32, WQ = FB == kMmE2m1Bf;
  constexpr bool SA = mm_scaled(FA), SB = mm_scaled(FB);
  constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
  constexpr int Q = MX ? KS / 64 : F32 ? 4 : 4;       // sub-steps of a slice
  constexpr int NS = FA == kMmF32Split ? 3 : 1;       // bf16 parts of a row's element
  constexpr int PA = FA == kMmE4m3 || FA == kMmF32Split ? 2 : 1;  // 16-byte pieces of a fragment
  constexpr int SBYTES = MX ? Q : 1;                  // a lane's scales of a slice
  constexpr int LA = Z::LA, LB = Z::LB;
  constexpr int ESA = mm_bits(FA) / 8, ESB = mm_bits(FB) / 8;  // 0 for e2m1
  static_assert(WTM % 32 == 0 && WTN % 32 == 0 && Q % 2 == 0, "tile shape");
  static_assert(S * STAGE <= 156 * 1024 && (S - 1) * (LA + LB) < 64, "ring");
  static_assert(!TA || FA == kMmBf16 || FA == kMmF32, "transposed rows");
  static_assert(!TB || FB == kMmBf16 || FB == kMmF32, "transposed matrix");
  static_assert(!TA || RBA % 256 == 0, "transposing reads take whole 256-byte windows");
  static_assert(!TB || RBB % 256 == 0, "transposing reads take whole 256-byte windows");
  // One object per slot, so that reads of one are known not to touch another.
  __shared__ __attribute__((aligned(1024))) char ring0[STAGE];
  __shared__ __attribute__((aligned(1024))) char ring1[STAGE];
  __shared__ __attribute__((aligned(1024))) char ring2[S > 2 ? STAGE : 16];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 31, fg = lane >> 5;
  const int wm = (wid / WN) * WTM, wn = (wid % WN) * WTN;
  const int nt = (p.N + BN - 1) / BN;

  // ---- the block's tile.  Blocks go to the 8 XCDs round robin: XCD x takes
  // the x-th eighth of the tiles, in groups of GM row tiles, column by column,
  // so that blocks running together share rows and matrix panels in its L2.
  constexpr int GM = 8;
  int e, row0, rows, n0, KT, krow0 = 0, K = p.K;
  {
    const int x = blockIdx.x & 7, j = blockIdx.x >> 3;
    int mt, col;
    if constexpr (TN_) {
      const int mts = (p.M + BM - 1) / BM, per_e = mts * nt;
      const int share = (per_e + 7) >> 3;  // of an expert's tiles
      e = j / share;
      const int t = x * share + (j - e * share);
      if (e >= p.E || t >= per_e) return;
      const int first = t / (GM * nt) * GM, in = t - first * nt;
      const int gsz = mts - first < GM ? mts - first : GM;
      mt = first + in % gsz;
      col = in / gsz;
      row0 = mt * BM;
      rows = p.M - row0 < BM ? p.M - row0 : BM;
      int o0 = 0, o1 = int(p.R);
      if (p.offsets != nullptr) {
        o0 = offset_at(p.offsets, e, p.E, p.R);
        o1 = offset_at(p.offsets, e + 1, p.E, p.R);
      }
      krow0 = __builtin_amdgcn_readfirstlane(o0);
      K = __builtin_amdgcn_readfirstlane(o1 > o0 ? o1 - o0 : 0);
    } else {
      int o[5], incl = 0, last = 0, mts;
      if (p.offsets != nullptr) mts = row_tiles<BM>(p.offsets, p.E, p.R, lane, o, incl, last);
      else mts = int((p.R + BM - 1) / BM);
      const int total = mts * nt, share = (total + 7) >> 3;  // at most the grid
      const int t = x * share + j;
      if (j >= share || t >= total) return;
      const int first = t / (GM * nt) * GM, in = t - first * nt;
      const int gsz = mts - first < GM ? mts - first : GM;
      mt = first + in % gsz;
      col = in / gsz;
      if (p.offsets != nullptr) {
        const RowTile r = row_tile<BM>(mt, o, incl, last, p.E, p.R, lane);
        e = r.e;
        row0 = r.row0;
        rows = r.rows;
      } else {
        e = 0;
        row0 = mt * BM;
        rows = p.R - row0 < BM ? int(p.R - row0) : BM;
      }
    }
    n0 = __builtin_amdgcn_readfirstlane(col * BN);
    e = __builtin_amdgcn_readfirstlane(e);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(rows);
    KT = (K + KS - 1) / KS;
    if (!TN_ && e == p.E && p.offsets != nullptr) KT = 0;  // rows of no expert
  }
  const int cols = p.N - n0 < BN ? p.N - n0 : BN;

  // ---- load sources: scalar bases and the lanes' offsets from them
  const int64_t pitch_a = TA ? p.lda * ESA : p.lda * mm_bits(FA) / 8;
  const int64_t pitch_b = TN_ ? p.ldb * ESB
                              : TB ? int64_t(p.N) * ESB : int64_t(p.K) * mm_bits(FB) / 8;
  const char* base_a = static_cast<const char*>(p.A);
  const char* base_b = static_cast<const char*>(p.B);
  if constexpr (TA) base_a += krow0 * pitch_a + int64_t(row0) * ESA;
  else base_a += row0 * pitch_a;
  if constexpr (TN_) base_b += krow0 * pitch_b + int64_t(n0) * ESB;
  else if constexpr (TB) base_b += int64_t(e) * p.K * pitch_b + int64_t(n0) * ESB;
  else base_b += (int64_t(e) * p.N + n0) * pitch_b;
  base_a = scalar_ptr(base_a);
  base_b = scalar_ptr(base_b);
  uint32_t off_a[LA], off_b[LB];
  // The lane's chunk of a row along K is the same in all its loads: NW loads on,
  // rows have moved by a multiple of the swizzle's period.
  const int chunk_a = ((lane * 16 % RBA) / 16) ^ swz<RBA>((wid * 1024 + lane * 16) / RBA);
  const int chunk_b = ((lane * 16 % RBB) / 16) ^ swz<RBB>((wid * 1024 + lane * 16) / RBB);
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int at = (wid + NW * i) * 1024 + lane * 16, r = at / RBA, c = (at % RBA) / 16;
    if constexpr (TA) {
      const int ch = c ^ swz_t<mm_bits(FA)>(r);
      off_a[i] = ch * 16 < rows * ESA ? uint32_t(r * pitch_a) + ch * 16 : kBeyond;
    } else {
      off_a[i] = uint32_t(r * pitch_a) + chunk_a * 16;
    }
  }
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int at = (wid + NW * i) * 1024 + lane * 16, r = at / RBB, c = (at % RBB) / 16;
    if constexpr (TB) {
      const int ch = c ^ swz_t<mm_bits(FB)>(r);
      off_b[i] = ch * 16 < cols * ESB ? uint32_t(r * pitch_b) + ch * 16 : kBeyond;
    } else {
      off_b[i] = uint32_t(r * pitch_b) + chunk_b * 16;
    }
  }
  // Slice kt into a slot; one past the last is all zeros (an empty buffer), so
  // that the loop has no special cases.  Across K the slice's last row ends
  // the buffer; along K lanes past K load from beyond it.
  auto issue = [&](int kt, char* slot) {
    const int left = K - kt * KS > 0 ? K - kt * KS : 0;  // elements
    const int take = left < KS ? left : KS;
    const uint32_t rec_a =
        TA ? uint32_t((take - 1) * pitch_a + rows * ESA)
           : uint32_t((rows - 1) * pitch_a) + uint32_t(int64_t(left) * mm_bits(FA) / 8);
    const uint32_t rec_b =
        TB ? uint32_t((take - 1) * pitch_b + cols * ESB)
           : uint32_t((cols - 1) * pitch_b) + uint32_t(int64_t(left) * mm_bits(FB) / 8);
    const auto ra = buffer(base_a + (TA ? kt * KS * pitch_a : int64_t(kt) * RBA), left ? rec_a : 0u);
    const auto rb = buffer(base_b + (TB ? kt * KS * pitch_b : int64_t(kt) * RBB), left ? rec_b : 0u);
    const bool in_a = TA || chunk_a * 128 < take * mm_bits(FA);
    const bool in_b = TB || chunk_b * 128 < take * mm_bits(FB);
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int blk = wid + NW * i;
      if (Z::ABYTES / 1024 % NW != 0 && blk >= Z::ABYTES / 1024) break;
      dma16(ra, slot + blk * 1024, in_a ? off_a[i] : kBeyond);
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int blk = wid + NW * i;
      if (Z::BBYTES / 1024 % NW != 0 && blk >= Z::BBYTES / 1024) break;
      dma16(rb, slot + Z::ABYTES + blk * 1024, in_b ? off_b[i] : kBeyond);
    }
  };

  // ---- scales: a lane's bytes of its rows and columns, fetched a slice ahead
  const int KB = p.K / 32;
  const uint8_t* sbase_a = nullptr;
  const uint8_t* sbase_b = nullptr;
  uint32_t soff_a[SA ? TM : 1], soff_b[SB ? TN : 1];
  if constexpr (SA) {
    sbase_a = reinterpret_cast<const uint8_t*>(
        scalar_ptr(reinterpret_cast<const char*>(p.As) + int64_t(row0) * KB));
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = wm + 32 * i + fr;
      soff_a[i] = uint32_t(r < rows ? r : rows - 1) * uint32_t(KB);
    }
  }
  if constexpr (SB) {
    sbase_b = reinterpret_cast<const uint8_t*>(
        scalar_ptr(reinterpret_cast<const char*>(p.Bs) + (int64_t(e) * p.N + n0) * KB));
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int c = wn + 32 * j + fr;
      soff_b[j] = uint32_t(c < cols ? c : cols - 1) * uint32_t(KB);
    }
  }
  uint32_t next_a[SA ? TM : 1], next_b[SB ? TN : 1];  // of the slice behind the current one
  uint32_t sc_a[SA ? TM : 1], sc_b[SB ? TN : 1];      // of the current one
  auto fetch_scales = [&](int kt) {
    const int kb = MX ? kt * (KS / 32) + fg * SBYTES : kt * 2 + fg;
    if constexpr (SA) {
#pragma unroll
      for (int i = 0; i < TM; ++i) next_a[i] = scale_bytes<SBYTES>(sbase_a + soff_a[i], kb, KB);
    }
    if constexpr (SB) {
#pragma unroll
      for (int j = 0; j < TN; ++j) next_b[j] = scale_bytes<SBYTES>(sbase_b + soff_b[j], kb, KB);
    }
  };
  auto take_scales = [&]() {
    if constexpr (SA) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
        sc_a[i] = MX ? next_a[i] : __float_as_uint(scale_f32(next_a[i]));
    }
    if constexpr (SB) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        sc_b[j] = MX ? next_b[j] : __float_as_uint(scale_f32(next_b[j]));
    }
  };

  // ---- fragments.  Sub-step q of a lane (fr, fg) of rows along K:
  //   its k are 16 q + 8 fg .. (bf16, fp32: 8 q + 4 fg ..), or, beside an e2m1
  //   matrix, 32 fg + 8 q .. (bf16), 32 (Q fg + q) .. (e2m1), so that a lane's
  //   16 bytes of e2m1 and its scales are together.  e4m3 instructions take
  //   bytes 16 fg .. of the two groups of 32 that lanes 0-31 and 32-63 scale.
  u32x4 fa[2][TM][PA], fb[2][TN];
  u32x4 raw_b[WQ ? TN : 1];
  auto load_a = [&](const char* slot, int q, int buf) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if constexpr (!TA) {
        const int r = wm + 32 * i + fr, z = swz<RBA>(fr);
        const char* row = slot + r * RBA;
        auto chunk = [&](int c) { return *reinterpret_cast<const u32x4*>(row + ((c ^ z) << 4)); };
        if constexpr (FA == kMmBf16) {
          fa[buf][i][0] = chunk(WQ ? 4 * fg + q : 2 * q + fg);
        } else if constexpr (FA == kMmF32) {
          fa[buf][i][0] = chunk(2 * q + fg);
        } else if constexpr (FA == kMmF32Split) {
          const int c = WQ ? 8 * fg + 2 * q : 4 * q + 2 * fg;
          fa[buf][i][0] = chunk(c);
          fa[buf][i][1] = chunk(c + 1);
        } else if constexpr (FA == kMmE4m3Bf) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(row + (((2 * fg + (q >> 1)) ^ z) << 4) +
                                                          8 * (q & 1));
          fa[buf][i][0] = u32x4{v.x, v.y, 0u, 0u};
        } else if constexpr (FA == kMmE4m3) {
          fa[buf][i][0] = chunk(2 * q + fg);
          fa[buf][i][1] = chunk(2 * (Q + q) + fg);
        } else {
          fa[buf][i][0] = chunk(Q * fg + q);
        }
      } else if constexpr (FA == kMmBf16) {
        const int g = lane >> 4, l = lane & 15, u = ((wm / 32 + i) ^ (l >> 2)) * 64;
        const char* at = slot + (16 * q + 8 * fg + (l >> 2)) * RBA + u + (g & 1) * 32 + (l & 3) * 8;
        const u32x2 a = read_tr(at), b = read_tr(at + 4 * RBA);
        fa[buf][i][0] = u32x4{a.x, a.y, b.x, b.y};
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int k = 8 * q + 4 * fg + s, c = (wm + 32 * i + fr) * 4;
          fa[buf][i][0][s] = *reinterpret_cast<const uint32_t*>(
              slot + k * RBA + (c ^ (swz_t<32>(k) << 4)));
        }
      }
    }
  };
  auto load_b = [&](const char* slot0, int q, int buf) {
    const char* slot = slot0 + Z::ABYTES;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if constexpr (!TB) {
        const int r = wn + 32 * j + fr, z = swz<RBB>(fr);
        const char* row = slot + r * RBB;
        auto chunk = [&](int c) { return *reinterpret_cast<const u32x4*>(row + ((c ^ z) << 4)); };
        if constexpr (WQ) {
          if (q == 0) raw_b[j] = chunk(fg);
        } else if constexpr (MX) {
          fb[buf][j] = chunk(Q * fg + q);
        } else {
          fb[buf][j] = chunk(2 * q + fg);
        }
      } else if constexpr (FB == kMmBf16) {
        const int g = lane >> 4, l = lane & 15, u = ((wn / 32 + j) ^ (l >> 2)) * 64;
        const char* at = slot + (16 * q + 8 * fg + (l >> 2)) * RBB + u + (g & 1) * 32 + (l & 3) * 8;
        const u32x2 a = read_tr(at), b = read_tr(at + 4 * RBB);
        fb[buf][j] = u32x4{a.x, a.y, b.x, b.y};
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int k = 8 * q + 4 * fg + s, c = (wn + 32 * j + fr) * 4;
          fb[buf][j][s] = *reinterpret_cast<const uint32_t*>(
              slot + k * RBB + (c ^ (swz_t<32>(k) << 4)));
        }
      }
    }
  };
  auto convert_b = [&](int q, int buf) {  // e2m1 to bf16
    if constexpr (WQ) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        fb[buf][j] = bf16_of_e2m1x8(raw_b[j][q], __uint_as_float(sc_b[j]));
    }
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  auto mma = [&](auto qc, int buf) {
    constexpr int q = decltype(qc)::value;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      u32x4 part[NS];
      if constexpr (FA == kMmF32Split) split3(fa[buf][i][0], fa[buf][i][PA - 1], part);
      else if constexpr (FA == kMmE4m3Bf)
        part[0] = bf16_of_e4m3x8(fa[buf][i][0][0], fa[buf][i][0][1], __uint_as_float(sc_a[i]));
      else part[0] = fa[buf][i][0];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if constexpr (MX) {
          acc[i][j] = mfma_mx<FA == kMmE4m3 ? 0 : 4, q>(fa[buf][i][0], fa[buf][i][PA - 1],
                                                        fb[buf][j], acc[i][j], sc_a[i], sc_b[j]);
        } else if constexpr (F32) {
          acc[i][j] = mfma_f32(part[0], fb[buf][j], acc[i][j]);
        } else {
          // the smallest part first
#pragma unroll
          for (int s = NS - 1; s >= 0; --s) acc[i][j] = mfma_bf16(part[s], fb[buf][j], acc[i][j]);
        }
      }
    }
  };
  // One slice, read from `cur`; the fragments of the next one's first sub-step
  // come from `nxt` under the last one's matrix instructions.
  auto step = [&](int kt, char* cur, const char* nxt) {
    if constexpr (SA || SB) fetch_scales(kt + 1 < KT ? kt + 1 : kt);
    auto sub = [&](auto qc) {
      constexpr int q = decltype(qc)::value;
      if constexpr (q + 1 < Q) {
        load_a(cur, q + 1, (q + 1) & 1);
        load_b(cur, q + 1, (q + 1) & 1);
        convert_b(q + 1, (q + 1) & 1);
        mma(qc, q & 1);
      } else {
        wait_loads<(S - 2) * Z::LMIN>();
        slot_barrier();
        issue(kt + S, cur);
        load_a(nxt, 0, 0);
        load_b(nxt, 0, 0);
        mma(qc, q & 1);
        take_scales();
        convert_b(0, 0);
      }
    };
    sub(std::integral_constant<int, 0>{});
    sub(std::integral_constant<int, 1>{});
    if constexpr (Q == 4) {
      sub(std::integral_constant<int, 2>{});
      sub(std::integral_constant<int, 3>{});
    }
  };
  if (KT > 0) {
    issue(0, ring0);
    issue(1, ring1);
    if constexpr (S > 2) issue(2, ring2);
    if constexpr (SA || SB) fetch_scales(0);
    wait_loads<(S - 1) * Z::LMIN>();
    slot_barrier();
    load_a(ring0, 0, 0);
    load_b(ring0, 0, 0);
    take_scales();
    convert_b(0, 0);
    int kt = 0;
    for (; kt + S <= KT; kt += S) {
      step(kt, ring0, ring1);
      if constexpr (S == 2) {
        step(kt + 1, ring1, ring0);
      } else {
        step(kt + 1, ring1, ring2);
        step(kt + 2, ring2, ring0);
      }
    }
    if (kt < KT) step(kt, ring0, ring1);
    if constexpr (S > 2) {
      if (kt + 1 < KT) step(kt + 1, ring1, ring2);
    }
    wait_loads<0>();  // no load into LDS outlives the block
  }

  // ---- epilogue: lane (fr, fg), register v holds row 8 (v / 4) + 4 fg + v % 4,
  // column fr of a 32 x 32 piece; four rows of a column are transposed inside a
  // lane quad, so that a lane stores four columns of a row.
  const int q4 = fr & 3, cl = wn + (fr & ~3);
  OT* out = static_cast<OT*>(p.C);
  const int64_t ldc = TN_ ? p.N : p.ldc;
  const int64_t first = TN_ ? int64_t(e) * p.M + row0 : int64_t(row0);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int vq = 0; vq < 4; ++vq) {
      const int r = wm + 32 * i + 8 * vq + 4 * fg + q4;
      OT* o = out + (first + r) * ldc + n0 + cl;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        float b[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) b[w] = acc[i][j][4 * vq + w];
        quad_transpose(b, q4);
        if (r < rows && cl + 32 * j < cols) store4<OT>(o + 32 * j, b);
      }
    }
  }
}

template <int LAYOUT, int FA, int FB, typename OT, int BM, int BN, int WM, int WN, int S>
hipError_t launch_tile(const MmParams& p, const Launch& s) {
  const int64_t nt = (p.N + BN - 1) / BN;
  int64_t grid;
  if (LAYOUT == kMmTN) {
    grid = 8 * int64_t(p.E) * (((p.M + BM - 1) / BM * nt + 7) / 8);
  } else {
    // row tiles at most: every expert's last one, and that of the rows of none, may be partial
    const int64_t full = p.R / BM, parts = p.offsets == nullptr ? 1 : int64_t(p.E) + 1;
    const int64_t mts = full + (parts < p.R ? parts : p.R);
    grid = (mts * nt + 7) / 8 * 8;
  }
  if (grid <= 0) return hipSuccess;
  if (grid * (64 * WM * WN) > 0x7fffffff) return hipErrorInvalidValue;
  return launch_kernel(mm_kernel<LAYOUT, FA, FB, OT, BM, BN, WM, WN, S>, dim3(unsigned(grid)),
                       dim3(64 * WM * WN), 0, s, p);
}

}  // namespace mm
}  // namespace topmoe
