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
//                  by truncation, exact from 2^-110 on; three bf16 instructions
//                  instead of eight fp32 ones at a sixteenth of the rate
//   e2m1 matrix beside bf16 rows: 16 bytes of a lane are its 32 k of a slice,
//                  turned into bf16 with their scale (exact below 2^128) as they
//                  are used
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

// The descriptor of `bytes` bytes from p on; both uniform.
__device__ __forceinline__ u32x4 buffer(const char* p, uint32_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return u32x4{uint32_t(v), uint32_t(v >> 32) & 0xffffu, bytes, 0x00020000u};
}
// 16 bytes a lane into LDS, lane i's at lds + 16 i; out of a lane's bounds: zeros.
// In assembly: of loads into LDS that it knows the compiler waits for all before
// a transposing read, and before a read of LDS that they do not write.  So the
// waits are this code's own: wait_loads and slot_barrier before a slot is read.
// (The clobber of m0 is meant: the compiler sets it right before each own use.
// One wait state between the write of m0 and its use, five between a vector
// instruction that wrote the descriptor, a readfirstlane say, and its use.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(u32x4 r, uint32_t lds, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(off), "s"(r) : "memory", "m0");
}
// The same of 4 bytes a lane, lane i's at lds + 4 i.
__device__ __forceinline__ void dma4(u32x4 r, uint32_t lds, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(lds), "v"(off), "s"(r) : "memory", "m0");
}
#pragma clang diagnostic pop
__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)p));
}
template <typename T>
__device__ __forceinline__ __attribute__((address_space(3))) T* lds_at(uint32_t at) {
  return reinterpret_cast<__attribute__((address_space(3))) T*>(at);
}
__device__ __forceinline__ u32x2 read_tr(uint32_t at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_at<s16x4>(at)));
}
// a's odd rows of 16 lanes change places with b's even ones; in each row of 16
// lanes a's upper 8 lanes with b's lower 8.
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap8(uint32_t& a, uint32_t& b) {
  const uint32_t x = a;  // row_ror:8 into the upper, into the lower banks
  a = __builtin_amdgcn_update_dpp(x, b, 0x128, 0xf, 0xc, false);
  b = __builtin_amdgcn_update_dpp(b, x, 0x128, 0xf, 0x3, false);
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
// e2m1 by a format FY: 0 e4m3 (eight registers), 4 e2m1 (four); byte SEL of the
// scales.  In assembly: through the builtin the compiler keeps the accumulators
// apart from the results, about 100 registers more, which spill.  So the waits
// are this code's own: two states between a vector instruction that wrote an
// operand and this one, and settle() before anything but another of these reads
// or writes an accumulator.
template <int FY, int SEL>
__device__ __forceinline__ void mfma_mx(u32x4 a, u32x4 b0, u32x4 b1, f32x16& c, uint32_t sa,
                                        uint32_t sb) {
  if constexpr (FY == 4) {
    if constexpr (SEL == 0)
      asm("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
          : "+v"(c) : "v"(a), "v"(b0), "v"(sa), "v"(sb));
    else if constexpr (SEL == 1)
      asm("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
          : "+v"(c) : "v"(a), "v"(b0), "v"(sa), "v"(sb));
    else if constexpr (SEL == 2)
      asm("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[1,1,0] cbsz:4 blgp:4"
          : "+v"(c) : "v"(a), "v"(b0), "v"(sa), "v"(sb));
    else
      asm("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[1,1,0] cbsz:4 blgp:4"
          : "+v"(c) : "v"(a), "v"(b0), "v"(sa), "v"(sb));
  } else {
    const i32x8 y = {int(b0[0]), int(b0[1]), int(b0[2]), int(b0[3]),
                     int(b1[0]), int(b1[1]), int(b1[2]), int(b1[3])};
    static_assert(SEL < 2, "two sub-steps");
    if constexpr (SEL == 0)
      asm("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[0,0,0] cbsz:4"
          : "+v"(c) : "v"(a), "v"(y), "v"(sa), "v"(sb));
    else
      asm("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4"
          : "+v"(c) : "v"(a), "v"(y), "v"(sa), "v"(sb));
  }
}
// Two e2m1 / e4m3 values times a scale as two bf16: exact, but infinite from 2^128
// on (e2m1 4 and 6 with the scale byte 253, 2 to 6 with 254; e4m3 from 247 on), and
// e4m3 with bytes below 3 rounded to multiples of 2^-133, bf16's smallest subnormal.
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
// Below 2^-110 the last part ends with bf16's subnormals: bits under 2^-133 are
// dropped.  An infinity is its own first part, with no rest; NaN leaves NaN in the
// rest.  (Parts that are 0 meet an infinite element of the matrix as NaN.)
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

// The offsets' expert e, held inside [0, R] so that no row outside is touched
// whatever the array holds; expert 0 starts at row 0.  No offsets: one expert.
__device__ __forceinline__ int offset_at(const int32_t* offsets, int e, int E, int64_t R) {
  if (e <= 0) return 0;
  if (offsets == nullptr) return int(R);
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

// The parts that an expert's `rows` are summed in, of `most` at most (0: one).
__device__ __forceinline__ int parts_of(int rows, int most) {
  return most > 0 && rows > most ? 1 + (rows - 1) / most : 1;
}
// (Up to 64 experts, one a lane.)  The expert and part that unit u is, longest
// parts first, so that the longest sums start first, and the number of the part
// among those that are kept apart; false past the last.
struct RowPart {
  int e, part, parts, slot;
};
__device__ __forceinline__ bool row_part(const int32_t* offsets, int E, int64_t R, int most, int u,
                                         int lane, RowPart& out) {
  const int rows = lane < E ? offset_at(offsets, lane + 1, E, R) - offset_at(offsets, lane, E, R)
                            : -1;
  const int parts = lane < E ? parts_of(rows, most) : 0;
  const int kept = parts > 1 ? parts : 0;
  const int slot = wave_inclusive_scan(kept, lane) - kept;
  int before;  // units of experts that come first
  if (!mm_tn_sorted(R, E)) {
    before = wave_inclusive_scan(parts, lane) - parts;
  } else {
    const int len = parts > 0 ? (rows + parts - 1) / parts : -1;
    before = 0;
    for (int e = 0; e < E; ++e) {
      const int other = __builtin_amdgcn_readlane(len, e), n = __builtin_amdgcn_readlane(parts, e);
      before += other > len || (other == len && e < lane) ? n : 0;
    }
  }
  const uint64_t m = __ballot(lane < E && u >= before && u < before + parts);
  if (m == 0) return false;
  const int at = __ffsll((long long)m) - 1;
  out.e = at;
  out.part = u - __builtin_amdgcn_readlane(before, at);
  out.parts = __builtin_amdgcn_readlane(parts, at);
  out.slot = __builtin_amdgcn_readlane(slot, at) + out.part;
  return out.parts == 1 || out.slot < mm_tn_parts(R, most, E);  // (offsets that do decrease)
}

// Elements of a K slice of Q sub-steps (an e2m1 matrix beside bf16 has four:
// a lane's 16 bytes).
constexpr int slice_of(int fa, int fb, int Q) {
  return Q * (fa == kMmF32 ? 8 : fb == kMmE2m1 ? 64 : 16);
}

template <int LAYOUT, int FA, int FB, typename OT, int BM, int BN, int WM, int WN, int Q, int S>
struct Shape {
  static constexpr int KS = slice_of(FA, FB, Q);
  static constexpr bool TA = LAYOUT == kMmTN, TB = LAYOUT != kMmNT;  // rows across K
  static constexpr int RBA = TA ? BM * mm_bits(FA) / 8 : KS * mm_bits(FA) / 8;  // bytes of an LDS row
  static constexpr int RBB = TB ? BN * mm_bits(FB) / 8 : KS * mm_bits(FB) / 8;
  static constexpr int ABYTES = BM * KS * mm_bits(FA) / 8, BBYTES = BN * KS * mm_bits(FB) / 8;
  static constexpr int STAGE = ABYTES + BBYTES;
  // and the scales' tail, four bytes a row or column
  static constexpr int SROWS = (mm_scaled(FA) ? BM : 0) + (mm_scaled(FB) ? BN : 0);
  static constexpr int SLOT = STAGE + SROWS * 4;
  static constexpr int NW = WM * WN;
  static constexpr int LA = (ABYTES / 1024 + NW - 1) / NW, LB = (BBYTES / 1024 + NW - 1) / NW;
  static constexpr int LS = (SROWS / 64 + NW - 1) / NW;
  // two blocks a CU where their rings fit, else one
  static constexpr int WAVES = (2 * S * SLOT <= 160 * 1024 ? 2 : 1) * (NW > 4 ? NW / 4 : 1);  // a SIMD
  static constexpr int LMIN =  // fewest loads of a wavefront
      ABYTES / 1024 / NW + BBYTES / 1024 / NW + SROWS / 64 / NW;
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

// W: the scales of a row lie at multiples of four bytes.
template <int LAYOUT, int FA, int FB, typename OT, int BM, int BN, int WM, int WN, int Q, int S,
          bool W>
__global__ __launch_bounds__(64 * WM * WN, (Shape<LAYOUT, FA, FB, OT, BM, BN, WM, WN, Q, S>::WAVES))
void mm_kernel(MmParams p) {
  using Z = Shape<LAYOUT, FA, FB, OT, BM, BN, WM, WN, Q, S>;
  constexpr int KS = Z::KS, NW = Z::NW, RBA = Z::RBA, RBB = Z::RBB, STAGE = Z::STAGE;
  constexpr bool TA = Z::TA, TB = Z::TB, TN_ = LAYOUT == kMmTN;
  constexpr bool MX = FB == kMmE2m1, F32 = FA == kMmF32, WQ = FB == kMmE2m1Bf;
  constexpr bool SA = mm_scaled(FA), SB = mm_scaled(FB);
  constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
  constexpr int NS = FA == kMmF32Split ? 3 : 1;       // bf16 parts of a row's element
  constexpr int PA = FA == kMmE4m3 || FA == kMmF32Split ? 2 : 1;  // 16-byte pieces of a fragment
  constexpr int SBYTES = MX ? Q : 1;                  // a lane's scales of a slice
  constexpr int LA = Z::LA, LB = Z::LB;
  constexpr int ESA = mm_bits(FA) / 8, ESB = mm_bits(FB) / 8;  // 0 for e2m1
  static_assert(WTM % 32 == 0 && WTN % 32 == 0 && (Q == 2 || Q == 4) && (!WQ || Q == 4), "tile shape");
  static_assert(!(SA || SB) || KS == 128 || KS == 64, "scales of a slice");
  static_assert(!(SA || SB) || (BM % 64 == 0 && BN % 64 == 0), "a load's scales are one operand's");
  static_assert((S == 3 || S == 4) && S * Z::SLOT <= 160 * 1024 && (S - 1) * (LA + LB + Z::LS) < 64,
                "ring");
  static_assert(W || Z::SROWS / 64 < NW, "loads of scales are counted as loads into LDS");
  static_assert(!TA || FA == kMmBf16 || FA == kMmF32, "transposed rows");
  static_assert(!TB || FB == kMmBf16 || FB == kMmF32, "transposed matrix");
  static_assert(!TA || RBA % 256 == 0, "transposing reads take whole 256-byte windows");
  static_assert(!TB || RBB % 256 == 0, "transposing reads take whole 256-byte windows");
  __shared__ __attribute__((aligned(1024))) char slots[S * Z::SLOT];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 31, fg = lane >> 5;
  // The matrix's column that a lane loads, of 32: bits 2 and 3 of fr in turn, so
  // that a lane's results are runs of eight columns.
  const int fc = (fr & 0x13) | (fr & 4) << 1 | (fr & 8) >> 1;
  const int wm = (wid / WN) * WTM, wn = (wid % WN) * WTN;
  const int nt = (p.N + BN - 1) / BN;
  const int64_t pitch_a = TA ? p.lda * ESA : p.lda * mm_bits(FA) / 8;
  const int64_t pitch_b = TN_ ? p.ldb * ESB
                              : TB ? int64_t(p.N) * ESB : int64_t(p.K) * mm_bits(FB) / 8;

  // ---- the block's tiles.  Blocks go to the 8 XCDs round robin.  NT, NN: XCD x
  // takes the x-th eighth of the tiles, in groups of GM row tiles, column by
  // column, so that blocks running together share rows and matrix panels in its
  // L2, and the grid's blocks of an XCD take its tiles in turn.  TN, where an
  // expert's rows are the length of its tiles: a block a tile; each XCD takes an
  // eighth of every expert's tiles (or of each of its parts'), so that the work is
  // even however the rows are spread.  Whole experts for an XCD read a third of the
  // bytes past the L2s (16384 tokens, top-2 of 8, 768 x 2432: 209 MB, of eighths
  // 634), which gained little and cost up to threefold (us, eighths and wholes):
  // E = 8, 768 x 2432, 32768 rows, alike 127 and 121, half of them one expert's 150
  // and 148; 1024 x 4096, 24576 rows in parts, a softmax of scale 0.7 227 and 268;
  // 4096 x 8192, 16384 rows whole, alike 980 and 990, half one expert's 1040 and 2840;
  // fp32 768 x 2432, 16384 rows, a third one expert's 497 and 730;  E = 16, 2048 x 1408,
  // 16384 rows, half one expert's 173 and 326.
  constexpr int GM = 8;
  struct Tile {
    const char *a, *b;          // first bytes of the tile's rows and columns
    const uint8_t *sa, *sb;     // and of their scales
    int e, row0, n0, rows, cols, K, KT;  // KT: slices, whole rounds of the ring
    int part;  // NN: the chunk of K; TN: the sum's number among the parts, or -1
  };
  const int xcd = blockIdx.x & 7, local = blockIdx.x >> 3;
  constexpr bool CHUNKS = LAYOUT == kMmNN && sizeof(OT) == 4;
  const int chunks = CHUNKS && p.kchunk > 0 ? (p.K + p.kchunk - 1) / p.kchunk : 1;
  int o[5], incl = 0, last = 0, mts, share, total, mine;
  const int blocks = gridDim.x >> 3;
  if constexpr (TN_) {
    mts = (p.M + BM - 1) / BM;
    total = mts * nt;
    share = (total + 7) >> 3;
    const int end = share * int(mm_tn_units(p.R, p.most, p.E));
    mine = local < end ? (end - local + blocks - 1) / blocks : 0;
  } else {
    if (p.offsets != nullptr) mts = row_tiles<BM>(p.offsets, p.E, p.R, lane, o, incl, last);
    else mts = int((p.R + BM - 1) / BM);
    total = mts * nt * chunks;  // at most the tiles the grid was planned for
    share = (total + 7) >> 3;
    const int end = total - xcd * share < share ? total - xcd * share : share;
    mine = local < end ? (end - local + blocks - 1) / blocks : 0;
  }
  mine = __builtin_amdgcn_readfirstlane(mine);
  // opaque: of a loop known to run once the compiler keeps 80 registers more
  asm volatile("" : "+s"(mine));
  if (mine <= 0) return;
  auto tile = [&](int i) {
    Tile t;
    int at;
    t.part = 0;
    RowPart rp{};
    bool any = true;  // TN: there is such a unit and tile
    if constexpr (TN_) {
      const int n = local + i * blocks, unit = n / share;
      at = n - unit * share + xcd * share;
      any = at < total;
      if (p.E > kMmPartExperts) {  // one after the other, each whole
        rp = RowPart{unit, 0, 1, 0};
        any = any && unit < p.E;
      } else {
        any = row_part(p.offsets, p.E, p.R, p.most, unit, lane, rp) && any;
      }
      at = any ? at : 0;
      t.part = rp.parts > 1 ? rp.slot : -1;
    } else {
      at = xcd * share + local + i * blocks;
      if constexpr (CHUNKS) {
        t.part = at / (mts * nt);
        at -= t.part * (mts * nt);
      }
    }
    t.part = __builtin_amdgcn_readfirstlane(t.part);
    const int first = at / (GM * nt) * GM, in = at - first * nt;
    const int gsz = mts - first < GM ? mts - first : GM;
    const int mt = first + in % gsz;
    t.n0 = __builtin_amdgcn_readfirstlane(in / gsz * BN);
    t.cols = p.N - t.n0 < BN ? p.N - t.n0 : BN;
    int krow0 = 0;
    if constexpr (TN_) {
      t.e = __builtin_amdgcn_readfirstlane(rp.e);
      t.row0 = mt * BM;
      t.rows = !any ? 0 : p.M - t.row0 < BM ? p.M - t.row0 : BM;
      const int o0 = offset_at(p.offsets, t.e, p.E, p.R);
      const int o1 = offset_at(p.offsets, t.e + 1, p.E, p.R);
      const int n = any && o1 > o0 ? o1 - o0 : 0, len = any ? (n + rp.parts - 1) / rp.parts : 0;
      const int left = n - rp.part * len;
      krow0 = __builtin_amdgcn_readfirstlane(o0 + rp.part * len);
      t.K = __builtin_amdgcn_readfirstlane(left < len ? (left > 0 ? left : 0) : len);
    } else if (p.offsets != nullptr) {
      const RowTile r = row_tile<BM>(mt, o, incl, last, p.E, p.R, lane);
      t.e = __builtin_amdgcn_readfirstlane(r.e);
      t.row0 = r.row0;
      t.rows = r.rows;
      t.K = t.e == p.E ? 0 : p.K;  // rows of no expert: a product over nothing
    } else {
      t.e = 0;
      t.row0 = mt * BM;
      t.rows = p.R - t.row0 < BM ? int(p.R - t.row0) : BM;
      t.K = p.K;
    }
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    if constexpr (CHUNKS) {
      if (p.kchunk > 0) {
        krow0 = t.part * p.kchunk;
        t.K = t.K - krow0 < p.kchunk ? (t.K > krow0 ? t.K - krow0 : 0) : p.kchunk;
      }
    }
    const int slices = (t.K + KS - 1) / KS;
    t.KT = slices > S ? (slices + S - 1) / S * S : S;
    t.a = static_cast<const char*>(p.A);
    t.b = static_cast<const char*>(p.B);
    if constexpr (TA) t.a += krow0 * pitch_a + int64_t(t.row0) * ESA;
    else t.a += t.row0 * pitch_a + int64_t(krow0) * mm_bits(FA) / 8;
    if constexpr (TN_) t.b += krow0 * pitch_b + int64_t(t.n0) * ESB;
    else if constexpr (TB) t.b += (int64_t(t.e) * p.K + krow0) * pitch_b + int64_t(t.n0) * ESB;
    else t.b += (int64_t(t.e) * p.N + t.n0) * pitch_b;
    t.sa = SA ? p.As + int64_t(t.row0) * (p.K / 32) : nullptr;
    t.sb = SB ? p.Bs + (int64_t(t.e) * p.N + t.n0) * (p.K / 32) : nullptr;
    return t;
  };

  // ---- loads.  Wavefront w fills the 1 KB blocks w, w + NW, ... of each
  // operand's part of a slot; a lane's 16-byte chunk of the LDS row is the same
  // in all of them (rows move by a multiple of the swizzle's period).
  const int row_a = (wid * 1024 + lane * 16) / RBA, row_b = (wid * 1024 + lane * 16) / RBB;
  const int chunk_a = ((lane * 16 % RBA) / 16) ^ (TA ? swz_t<mm_bits(FA)>(row_a) : swz<RBA>(row_a));
  const int chunk_b = ((lane * 16 % RBB) / 16) ^ (TB ? swz_t<mm_bits(FB)>(row_b) : swz<RBB>(row_b));
  static_assert(TA ? (mm_bits(FA) == 16 ? NW * 1024 / RBA % 4 == 0 : NW * 1024 / RBA % 8 == 0)
                   : NW * 4 % (RBA / 16) == 0, "one chunk a lane");
  static_assert(TB ? (mm_bits(FB) == 16 ? NW * 1024 / RBB % 4 == 0 : NW * 1024 / RBB % 8 == 0)
                   : NW * 4 % (RBB / 16) == 0, "one chunk a lane");
  const uint32_t ring = lds_address(slots);
  uint32_t off_a[LA], off_b[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i)
    off_a[i] = uint32_t((row_a + i * NW * 1024 / RBA) * pitch_a) + chunk_a * 16;
#pragma unroll
  for (int i = 0; i < LB; ++i)
    off_b[i] = uint32_t((row_b + i * NW * 1024 / RBB) * pitch_b) + chunk_b * 16;
  // Slice kt of a tile into a slot, in LA + LB loads, spread among the matrix
  // instructions; one past the tile's last is all zeros (an empty buffer).
  // Across K the slice's last row ends the buffer and lanes past the last
  // column load from beyond it; along K it ends with the last row, and lanes
  // past K load from beyond.
  struct Source {
    u32x4 ra, rb;
    bool in_a, in_b;
  };
  auto source = [&](const Tile& t, int kt) {
    const int left = t.K - kt * KS > 0 ? t.K - kt * KS : 0;  // elements
    const int take = left < KS ? left : KS;
    const uint32_t rec_a =
        TA ? uint32_t((take - 1) * pitch_a + t.rows * ESA)
           : uint32_t((t.rows - 1) * pitch_a) + uint32_t(int64_t(left) * mm_bits(FA) / 8);
    const uint32_t rec_b =
        TB ? uint32_t((take - 1) * pitch_b + t.cols * ESB)
           : uint32_t((t.cols - 1) * pitch_b) + uint32_t(int64_t(left) * mm_bits(FB) / 8);
    Source f;
    f.ra = buffer(t.a + (TA ? kt * KS * pitch_a : int64_t(kt) * RBA), left ? rec_a : 0u);
    f.rb = buffer(t.b + (TB ? kt * KS * pitch_b : int64_t(kt) * RBB), left ? rec_b : 0u);
    f.in_a = TA ? chunk_a * 16 < t.rows * ESA : chunk_a * 128 < take * mm_bits(FA);
    f.in_b = TB ? chunk_b * 16 < t.cols * ESB : chunk_b * 128 < take * mm_bits(FB);
    return f;
  };
  auto issue = [&](const Source& f, uint32_t slot, int l) {
    int w = wid;  // opaque, so that the slots' addresses are added up here, not kept
    asm volatile("" : "+s"(w));
    const int i = l < LA ? l : l - LA, blk = w + NW * i;
    if (l < LA) {
      if (Z::ABYTES / 1024 % NW == 0 || blk < Z::ABYTES / 1024)
        dma16(f.ra, slot + blk * 1024, f.in_a ? off_a[i] : kBeyond);
    } else {
      if (Z::BBYTES / 1024 % NW == 0 || blk < Z::BBYTES / 1024)
        dma16(f.rb, slot + Z::ABYTES + blk * 1024, f.in_b ? off_b[i] : kBeyond);
    }
  };
  // ---- scales: four bytes a row or column into the tail of the slice's slot,
  // the slice's (KS = 128) or those of its pair of slices (64); zeros (2^-127)
  // for rows past the tile's and, like all of the slice, past its K.  Scales
  // that do not lie at multiples of four bytes (!W) take ordinary loads and
  // stores, which wait for everything in flight.
  constexpr int SROWS = Z::SROWS, PER = KS / 32;
  auto issue_scales = [&](const Tile& t, int kt, uint32_t slot) {
    const int KB = p.K / 32, left = t.K / 32 - kt * PER, kb = PER == 4 ? 4 * kt : 2 * kt & ~3;
#pragma unroll
    for (int i = 0; i < Z::LS; ++i) {
      const int at = wid + NW * i;  // 64 rows or columns
      if (SROWS / 64 % NW != 0 && at >= SROWS / 64) break;
      const bool rows = SA && at < BM / 64;
      const int x0 = rows ? at * 64 : at * 64 - (SA ? BM : 0), n = rows ? t.rows : t.cols;
      const uint8_t* base = (rows ? t.sa : t.sb) + kb;
      const uint32_t to = slot + STAGE + at * 256;
      if constexpr (W) {
        const uint32_t bytes = left > 0 ? uint32_t(n) * uint32_t(KB) - uint32_t(kb) : 0u;
        dma4(buffer(reinterpret_cast<const char*>(base), bytes), to,
             uint32_t(x0 + lane) * uint32_t(KB));
      } else {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (x0 + lane < n && kb + j < t.K / 32)
            w |= uint32_t(base[uint32_t(x0 + lane) * uint32_t(KB) + j]) << (8 * j);
        *lds_at<uint32_t>(to + lane * 4) = w;
      }
    }
  };
  auto issue_all = [&](const Tile& t, int kt, uint32_t slot) {
    const Source f = source(t, kt);
#pragma unroll
    for (int l = 0; l < LA + LB; ++l) issue(f, slot, l);
    if constexpr (Z::SROWS > 0) issue_scales(t, kt, slot);
  };
  uint32_t sc_a[SA ? TM : 1], sc_b[SB ? TN : 1];  // of the current slice
  uint32_t nx_a[SA ? TM : 1], nx_b[SB ? TN : 1];  // of the next one
  auto read_scales = [&](uint32_t slot, int kt) {  // of slice kt
    typedef typename std::conditional<SBYTES == 2, uint16_t, uint8_t>::type word;
    const uint32_t at = slot + STAGE + fg * SBYTES + (PER == 2 ? 2 * (kt & 1) : 0);
    if constexpr (SA) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
        nx_a[i] = *lds_at<const word>(at + (wm + fr) * 4 + 128 * i);
    }
    if constexpr (SB) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        nx_b[j] = *lds_at<const word>(at + (wn + fc + (SA ? BM : 0)) * 4 + 128 * j);
    }
  };
  auto take_scales = [&]() {
    if constexpr (SA) {
#pragma unroll
      for (int i = 0; i < TM; ++i) sc_a[i] = MX ? nx_a[i] : __float_as_uint(scale_f32(nx_a[i]));
    }
    if constexpr (SB) {
#pragma unroll
      for (int j = 0; j < TN; ++j) sc_b[j] = MX ? nx_b[j] : __float_as_uint(scale_f32(nx_b[j]));
    }
  };

  // ---- fragments.  Sub-step q of a lane (fr, fg) of rows along K:
  //   its k are 16 q + 8 fg .. (bf16, fp32: 8 q + 4 fg ..), or, beside an e2m1
  //   matrix, 32 fg + 8 q .. (bf16), 32 (Q fg + q) .. (e2m1), so that a lane's
  //   16 bytes of e2m1 and its scales are together.  e4m3 instructions take
  //   bytes 16 fg .. of the two groups of 32 that lanes 0-31 and 32-63 scale.
  u32x4 fa[2][TM][PA], fb[2][TN];
  u32x4 raw_b[WQ ? TN : 1];
  auto load_a = [&](uint32_t slot, int q, int buf, int i) {
    if constexpr (!TA) {
      const int z = swz<RBA>(fr);
      const uint32_t row = slot + (wm + fr) * RBA;
      auto chunk = [&](int c) {
        return *lds_at<const u32x4>(row + ((c ^ z) << 4) + 32 * i * RBA);
      };
      if constexpr (FA == kMmBf16) {
        fa[buf][i][0] = chunk(WQ ? 4 * fg + q : 2 * q + fg);
      } else if constexpr (FA == kMmF32) {
        fa[buf][i][0] = chunk(2 * q + fg);
      } else if constexpr (FA == kMmF32Split) {
        const int c = WQ ? 8 * fg + 2 * q : 4 * q + 2 * fg;
        fa[buf][i][0] = chunk(c);
        fa[buf][i][1] = chunk(c + 1);
      } else if constexpr (FA == kMmE4m3Bf) {
        const u32x2 v = *lds_at<const u32x2>(row + (((2 * fg + (q >> 1)) ^ z) << 4) + 8 * (q & 1) +
                                             32 * i * RBA);
        fa[buf][i][0] = u32x4{v.x, v.y, 0u, 0u};
      } else if constexpr (FA == kMmE4m3) {
        fa[buf][i][0] = chunk(2 * q + fg);
        fa[buf][i][1] = chunk(2 * (Q + q) + fg);
      } else {
        fa[buf][i][0] = chunk(Q * fg + q);
      }
    } else if constexpr (FA == kMmBf16) {
      const int g = lane >> 4, l = lane & 15, u = ((wm / 32 + i) ^ (l >> 2)) * 64;
      const uint32_t at = slot + (16 * q + 8 * fg + (l >> 2)) * RBA + u + (g & 1) * 32 + (l & 3) * 8;
      const u32x2 a = read_tr(at), b = read_tr(at + 4 * RBA);
      fa[buf][i][0] = u32x4{a.x, a.y, b.x, b.y};
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int k = 8 * q + 4 * fg + s, c = (wm + 32 * i + fr) * 4;
        fa[buf][i][0][s] = *lds_at<const uint32_t>(slot + k * RBA + (c ^ (swz_t<32>(k) << 4)));
      }
    }
  };
  auto load_b = [&](uint32_t slot0, int q, int buf, int j) {
    const uint32_t slot = slot0 + Z::ABYTES;
    if constexpr (!TB) {
      const int z = swz<RBB>(fc);
      const uint32_t row = slot + (wn + fc) * RBB;
      auto chunk = [&](int c) {
        return *lds_at<const u32x4>(row + ((c ^ z) << 4) + 32 * j * RBB);
      };
      if constexpr (WQ) {
        if (q == 0) raw_b[j] = chunk(fg);
      } else if constexpr (MX) {
        fb[buf][j] = chunk(Q * fg + q);
      } else {
        fb[buf][j] = chunk(2 * q + fg);
      }
    } else if constexpr (FB == kMmBf16) {
      const int g = lane >> 4, l = lane & 15, u = ((wn / 32 + j) ^ (l >> 2)) * 64;
      const uint32_t at = slot + (16 * q + 8 * fg + (l >> 2)) * RBB + u + (g & 1) * 32 +
                          (l & 1) * 16 + (l & 2) * 4;
      const u32x2 a = read_tr(at), b = read_tr(at + 4 * RBB);
      fb[buf][j] = u32x4{a.x, a.y, b.x, b.y};
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int k = 8 * q + 4 * fg + s, c = (wn + 32 * j + fc) * 4;
        fb[buf][j][s] = *lds_at<const uint32_t>(slot + k * RBB + (c ^ (swz_t<32>(k) << 4)));
      }
    }
  };
  auto convert_b = [&](int q, int buf, int j) {  // e2m1 to bf16
    if constexpr (WQ) fb[buf][j] = bf16_of_e2m1x8(raw_b[j][q], __uint_as_float(sc_b[j]));
  };
  // The loads of a sub-step's fragments in the order of their first use.
  auto load = [&](uint32_t slot, int q, int buf, int l) {
    if (l == 0) load_a(slot, q, buf, 0);
    else if (l <= TN) load_b(slot, q, buf, l - 1);
    else load_a(slot, q, buf, l - TN);
  };

  // The matrix's columns are the instructions' rows, so that a lane ends with
  // runs of columns of one row.
  f32x16 acc[TM][TN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  };
  u32x4 part[NS];  // of the row fragment in use
  auto mma = [&](auto qc, int buf, int i, int j) {
    constexpr int q = decltype(qc)::value;
    if (j == 0) {
      if constexpr (FA == kMmF32Split) split3(fa[buf][i][0], fa[buf][i][PA - 1], part);
      else if constexpr (FA == kMmE4m3Bf)
        part[0] = bf16_of_e4m3x8(fa[buf][i][0][0], fa[buf][i][0][1], __uint_as_float(sc_a[i]));
      else part[0] = fa[buf][i][0];
    }
    if constexpr (MX) {
      mfma_mx<FA == kMmE4m3 ? 0 : 4, q>(fb[buf][j], fa[buf][i][0], fa[buf][i][PA - 1], acc[i][j],
                                        sc_b[j], sc_a[i]);
    } else if constexpr (F32) {
      acc[i][j] = mfma_f32(fb[buf][j], part[0], acc[i][j]);
    } else {
      // the smallest part first
#pragma unroll
      for (int s = NS - 1; s >= 0; --s) acc[i][j] = mfma_bf16(fb[buf][j], part[s], acc[i][j]);
    }
  };
  // One slice, read from slot C, while slice `kt` of tile t goes into the slot
  // read before; the fragments of the next slice's first sub-step come from the
  // next slot under the last one's matrix instructions; `next`: its number.
  // The loads are spread over all sub-steps, so that wavefronts do not queue for
  // the address unit; those of the last come behind the wait and the barrier.
  // `stored`: the stores of a tile before may still be under way behind the
  // loads that are waited for.
  constexpr int NST = sizeof(OT) == 2 ? TM * TN * 2 : TM * TN * 4;  // stores of a whole tile
  constexpr int LAST_LOADS = LA + LB - (Q - 1) * (LA + LB) / Q;
  constexpr int WAIT = (S - 2) * Z::LMIN > LAST_LOADS ? (S - 2) * Z::LMIN - LAST_LOADS : 0;
  constexpr int WAIT_ST = WAIT + NST < 63 ? WAIT + NST : 63;
  auto step = [&](auto slot_number, const Tile& t, int kt, int next, bool stored) {
    constexpr int C = decltype(slot_number)::value;
    uint32_t cur = ring + C * Z::SLOT, nxt = ring + (C + 1) % S * Z::SLOT;
    const uint32_t free = ring + (C + S - 1) % S * Z::SLOT;
    // opaque, so that addresses are added up here and not kept for every slot,
    // which spilled 26 registers of 4-bit 256 x 256 tiles; 1 to 3 percent slower
    // where nothing spills
    if constexpr (MX) asm volatile("" : "+s"(cur), "+s"(nxt));
    const Source f = source(t, kt);
    auto sub = [&](auto qc) {
      constexpr int q = decltype(qc)::value, NM = TM * TN, NL = TM + TN;
      constexpr bool LAST = q + 1 == Q;
      constexpr int D0 = q * (LA + LB) / Q, ND = (q + 1) * (LA + LB) / Q - D0;
      if constexpr (LAST) {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (SROWS > 0) issue_scales(t, kt, free);
        if (stored) wait_loads<WAIT_ST>();
        else wait_loads<WAIT>();
        slot_barrier();
        if constexpr (SROWS > 0) read_scales(nxt, next);
      }
      // behind each matrix instruction a part of the other work
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        __builtin_amdgcn_sched_barrier(0);
        mma(qc, q & 1, m / TN, m % TN);
#pragma unroll
        for (int l = m * NL / NM; l < (m + 1) * NL / NM; ++l)
          load(LAST ? nxt : cur, LAST ? 0 : q + 1, (q + 1) & 1, l);
#pragma unroll
        for (int l = m * ND / NM; l < (m + 1) * ND / NM; ++l) issue(f, free, D0 + l);
        if constexpr (!LAST) {
#pragma unroll
          for (int j = m * TN / NM; j < (m + 1) * TN / NM; ++j) convert_b(q + 1, (q + 1) & 1, j);
        }
      }
      if constexpr (LAST) {
        if constexpr (SROWS > 0) take_scales();
#pragma unroll
        for (int j = 0; j < TN; ++j) convert_b(0, 0, j);
      }
    };
    sub(std::integral_constant<int, 0>{});
    sub(std::integral_constant<int, 1>{});
    if constexpr (Q == 4) {
      sub(std::integral_constant<int, 2>{});
      sub(std::integral_constant<int, 3>{});
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // Every scaled instruction has been issued, then at least the 19 states that
  // the longest of them takes, then the accumulators are read.
  auto settle = [&]() {
#pragma unroll
    for (int t = 0; t < 2 * TM * TN; ++t) {
      if (t == TM * TN) asm volatile("s_nop 15\n\ts_nop 15" : "+v"(acc[0][0]));
      asm volatile("" : "+v"(acc[t / TN % TM][t % TN]));
    }
  };

  // ---- a tile's results.  Lane (fr, fg), register 8 s + v of a 32 x 32 piece:
  // row fr, column 16 s + 8 fg + v.  Swaps of rows of 16 and of 8 lanes bring
  // 128 bytes of a row (64 of an odd bf16 piece) to the lanes of one store, 16
  // in each: whole lines, which are written once, and past the L2's, where the
  // rows and matrices of the tiles to come stay (bf16, 32768 rows, 768 -> 4864,
  // and 4-bit rows, 16384 of 2048 -> 6464: 267 and 148 us; through the L2's 294
  // and 174; halves of lines past them 301 and 161, through them 300 and 178).
  // `wide`: fp32 into the parts whatever the dtype (TN).
  auto put = [&](const Tile& t, auto whole_tile, void* C, int64_t first, bool wide) {
    constexpr bool whole = decltype(whole_tile)::value;
    const int64_t ldc = TN_ ? p.N : p.ldc;
    const int64_t start = first * ldc + t.n0;
    const int b8 = (lane >> 3) & 1, b16 = (lane >> 4) & 1;
    // a line of eight chunks of 16 bytes: w[a][b], of row fr, becomes that of row
    // (lane & 7) + 8 a + 16 b, the lane's bits b8 and b16 the a and b it had
    auto line = [&](uint32_t (&w)[2][2][4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int a = 0; a < 2; ++a) swap16(w[a][0][k], w[a][1][k]);
#pragma unroll
        for (int b = 0; b < 2; ++b) swap8(w[0][b][k], w[1][b][k]);
      }
    };
    auto words = [&](const f32x16& d, int s, uint32_t (&w)[4]) {  // eight bf16
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(d[8 * s + 2 * k]),
                                                   static_cast<__bf16>(d[8 * s + 2 * k + 1])});
    };
    auto store = [&](auto* o, const uint32_t (&w)[4]) {
      __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4*>(o));
    };
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if (sizeof(OT) == 4 || wide) {
          int r = wm + 32 * i + (lane & 7), c = wn + 32 * j + 16 * b16 + 8 * fg + 4 * b8;
          asm volatile("" : "+v"(r), "+v"(c));  // no address is kept for the whole block
          float* o = static_cast<float*>(C) + start + (uint32_t(r) * uint32_t(ldc) + uint32_t(c));
          uint32_t w[2][2][4];
#pragma unroll
          for (int v = 0; v < 16; ++v)
            w[(v >> 2) & 1][v >> 3][v & 3] = __float_as_uint(acc[i][j][v]);
          line(w);
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (whole || (r + 8 * h < t.rows && c < t.cols)) store(o + 8 * h * ldc, w[h & 1][h >> 1]);
        } else if (j % 2 == 0 && j + 1 < TN) {
          int r = wm + 32 * i + (lane & 7), c = wn + 32 * j + 32 * b8 + 16 * b16 + 8 * fg;
          asm volatile("" : "+v"(r), "+v"(c));
          bf16_t* o = static_cast<bf16_t*>(C) + start + (uint32_t(r) * uint32_t(ldc) + uint32_t(c));
          uint32_t w[2][2][4];
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int s = 0; s < 2; ++s) words(acc[i][j + a < TN ? j + a : j], s, w[a][s]);
          line(w);
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (whole || (r + 8 * h < t.rows && c < t.cols)) store(o + 8 * h * ldc, w[h & 1][h >> 1]);
        } else if (j % 2 == 0) {
          int r = wm + 32 * i + (lane & 15), c = wn + 32 * j + 16 * b16 + 8 * fg;
          asm volatile("" : "+v"(r), "+v"(c));
          bf16_t* o = static_cast<bf16_t*>(C) + start + (uint32_t(r) * uint32_t(ldc) + uint32_t(c));
          uint32_t w[2][4];
#pragma unroll
          for (int s = 0; s < 2; ++s) words(acc[i][j], s, w[s]);
#pragma unroll
          for (int k = 0; k < 4; ++k) swap16(w[0][k], w[1][k]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (whole || (r + 16 * h < t.rows && c < t.cols)) store(o + 16 * h * ldc, w[h]);
        }
      }
    }
  };

  // ---- the ring runs on from tile to tile: under a tile's last slices the
  // first ones of the next are loaded, and they arrive under its stores.
  Tile cur = tile(0);
#pragma unroll
  for (int s = 0; s + 1 < S; ++s) issue_all(cur, s, ring + s * Z::SLOT);
  wait_loads<(S - 2) * Z::LMIN>();
  slot_barrier();
  if constexpr (SROWS > 0) read_scales(ring, 0);
#pragma unroll
  for (int l = 0; l < TM + TN; ++l) load(ring, 0, 0, l);
  if constexpr (SROWS > 0) take_scales();
#pragma unroll
  for (int j = 0; j < TN; ++j) convert_b(0, 0, j);
  bool stored = false;
  for (int i = 0; i < mine; ++i) {
    Tile nxt = cur;
    if (i + 1 < mine) nxt = tile(i + 1);
    else nxt.K = 0;  // nothing is loaded any more
    clear();
    for (int kt = 0; kt < cur.KT; kt += S) {
      const bool over = kt + S >= cur.KT;
      const bool st = stored && kt == 0;
      Tile src = cur;
      if (over) src = nxt;
      const int at = over ? 0 : kt + S;
      constexpr std::integral_constant<int, 0> c0{};
      constexpr std::integral_constant<int, 1> c1{};
      constexpr std::integral_constant<int, 2> c2{};
      step(c0, cur, kt + S - 1, kt + 1, st);
      if constexpr (S == 3) {
        step(c1, src, at, kt + 2, false);
        step(c2, src, at + 1, at, false);
      } else {
        constexpr std::integral_constant<int, 3> c3{};
        step(c1, src, at, kt + 2, st);
        step(c2, src, at + 1, kt + 3, false);
        step(c3, src, at + 2, at, false);
      }
    }
    if constexpr (MX) settle();
    const bool whole = cur.rows == BM && cur.cols == BN;
    if constexpr (TN_) {
      const bool part = cur.part >= 0;
      put(cur, std::false_type{}, part ? static_cast<void*>(p.part) : p.C,
          int64_t(part ? cur.part : cur.e) * p.M + cur.row0, part);
    } else {
      const int64_t first = (CHUNKS ? cur.part * p.R : 0) + cur.row0;
      if (whole) put(cur, std::true_type{}, p.C, first, false);
      else put(cur, std::false_type{}, p.C, first, false);
      stored = whole;
    }
    cur = nxt;
  }
  wait_loads<0>();  // no load into LDS outlives the block
}

// Blocks of a kernel that are on the device at once, asked once per device.
template <typename K>
int resident(K kernel, int threads, int (&cached)[64]) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (cached[dev] == 0) {
    int cus = 0, per_cu = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        cus <= 0)
      cus = 256;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, kernel, threads, 0) != hipSuccess ||
        per_cu <= 0)
      per_cu = 1;
    cached[dev] = cus * per_cu;
  }
  return cached[dev];
}

template <int LAYOUT, int FA, int FB, typename OT, int BM, int BN, int WM, int WN, int Q, int S,
          bool W = true>
hipError_t launch_tile(const MmParams& p, const Launch& s) {
  using Z = Shape<LAYOUT, FA, FB, OT, BM, BN, WM, WN, Q, S>;
  const int64_t nt = (p.N + BN - 1) / BN;
  auto kernel = mm_kernel<LAYOUT, FA, FB, OT, BM, BN, WM, WN, Q, S, W>;
  int64_t grid;
  if (LAYOUT == kMmTN) {
    const int64_t units = mm_tn_units(p.R, p.most, p.E);
    const int64_t tiles = (p.M + BM - 1) / BM * nt;
    grid = 8 * units * ((tiles + 7) / 8);
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
  } else {
    // row tiles at most: every expert's last one, and that of the rows of none, may be partial
    const int64_t full = p.R / BM, parts = p.offsets == nullptr ? 1 : int64_t(p.E) + 1;
    const int64_t tiles = (full + (parts < p.R ? parts : p.R)) * nt * mm_chunks(p.K, p.kchunk);
    if (tiles > 0x7fffffff) return hipErrorInvalidValue;
    static int cached[64] = {};
    const int64_t cap = resident(kernel, 64 * Z::NW, cached) / 8 * 8;
    grid = (tiles + 7) / 8 * 8;
    if (grid > cap && cap >= 8) grid = cap;
  }
  if (grid <= 0) return hipSuccess;
  if (grid * (64 * Z::NW) > 0x7fffffff) return hipErrorInvalidValue;
  return launch_kernel(kernel, dim3(unsigned(grid)), dim3(64 * Z::NW), 0, s, p);
}

}  // namespace mm
}  // namespace topmoe
