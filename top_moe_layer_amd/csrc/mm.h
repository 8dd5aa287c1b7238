// Products of rows grouped by expert with each expert's matrix (mm_impl.h,
// mm_few.hip): what a launch needs, in elements unless said.
#pragma once

#include "kernels.h"

namespace topmoe {

// Number formats of the operands.  The e4m3 / e2m1 ones come with a scale byte
// (2^(byte - 127)) per 32 elements along the contracted dimension.
enum MmFmt {
  kMmBf16 = 0,
  kMmF32 = 1,       // fp32 matrix instructions
  kMmF32Split = 2,  // fp32 as three bf16 parts, beside a bf16 or e2m1 matrix
  kMmE4m3 = 3,      // 8-bit matrix instructions
  kMmE4m3Bf = 4,    // e4m3 turned into bf16
  kMmE2m1 = 5,      // 4-bit matrix instructions
  kMmE2m1Bf = 6,    // e2m1 turned into bf16
};
constexpr bool mm_scaled(int f) { return f >= kMmE4m3; }
constexpr int mm_bits(int f) {
  return f == kMmBf16 ? 16 : f == kMmF32 || f == kMmF32Split ? 32
         : f == kMmE4m3 || f == kMmE4m3Bf ? 8 : 4;
}

// C[r, n] = sum over k of A[r, k] B_e[n, k]      (kMmNT: B_e [N, K])
// C[r, n] = sum over k of A[r, k] B_e[k, n]      (kMmNN: B_e [K, N])
//   for the rows r of expert e; rows of no expert get zeros
// C_e[m, n] = sum over e's rows r of A[r, m] B[r, n]  (kMmTN: A [R, M], B [R, N])
enum MmLayout { kMmNT = 0, kMmNN = 1, kMmTN = 2 };

struct MmParams {
  const void* A;
  const void* B;
  const uint8_t* As;  // [R, K / 32]
  const uint8_t* Bs;  // [E, N, K / 32]
  void* C;
  const int32_t* offsets;  // [E + 1] or NULL: one expert, all rows
  int64_t R;
  int64_t lda, ldb, ldc;  // row pitches of A and C, and of B in TN (else B is dense)
  int E, M, N, K;         // M: TN only; K: NT and NN only
};

constexpr int kMmMaxExperts = 256;
constexpr int kMx4Group = 32;  // channels that share a scale

// Rows an expert has on average (the host does not know how they are spread),
// and tiles of BM x BN that they then make.
inline int64_t mm_rows_each(const MmParams& p) { return (p.R + p.E - 1) / p.E; }
inline int64_t mm_tiles(const MmParams& p, int64_t bm, int64_t bn) {
  const int64_t experts = p.E < p.R ? p.E : p.R;
  return (mm_rows_each(p) + bm - 1) / bm * experts * ((p.N + bn - 1) / bn);
}

hipError_t launch_mm_bf16(MmLayout layout, const MmParams& p, const Launch& s);
hipError_t launch_mm_f32(MmLayout layout, const MmParams& p, const Launch& s);
// NT with a matrix in 4 bits (B, Bs); fa: kMmBf16 (C bf16), kMmF32Split (C fp32),
// kMmE4m3 (C bf16), kMmE4m3Bf (C fp32), kMmE2m1 (either).
hipError_t launch_mm_mx4(int fa, bool out_bf16, const MmParams& p, const Launch& s);
hipError_t launch_mm_f32_by_bf16(const MmParams& p, const Launch& s);

// ---- 4-bit values (mx4.hip): q [R, C / 2], scale [R, ceil(C / 32)], dense
hipError_t launch_mx4_pack(const void* x, int64_t ldx, int64_t R, int64_t C, int dtype, uint8_t* q,
                           uint8_t* scale, const Launch& s);
hipError_t launch_mx4_unpack(const uint8_t* q, const uint8_t* scale, int64_t R, int64_t C,
                             int dtype, void* x, int64_t ldx, const Launch& s);

}  // namespace topmoe
