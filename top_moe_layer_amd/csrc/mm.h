// Products of rows grouped by expert with each expert's matrix (mm_impl.h,
// mm_few.h): what a launch needs, in elements unless said.
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
  // Sums in parts, added up by launch_mm_sum_chunks and _rows: NN over chunks of kchunk of K
  // (0: whole), C then being the parts [chunks, R, N] in fp32; TN over parts of
  // an expert's rows, of most rows each (0: whole), those of experts with more
  // than one going to part [.., M, N], expert by expert.
  int kchunk, most;
  float* part;
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

// TN: of one expert.
inline int64_t mm_tn_tiles(const MmParams& p, int64_t bm, int64_t bn) {
  return (p.M + bm - 1) / bm * ((p.N + bn - 1) / bn);
}

hipError_t launch_mm_bf16(MmLayout layout, const MmParams& p, const Launch& s);
hipError_t launch_mm_f32(MmLayout layout, const MmParams& p, const Launch& s);
// NT with a matrix in 4 bits (B, Bs); fa: kMmBf16 (C bf16), kMmF32Split (C fp32),
// kMmE4m3 (C bf16), kMmE4m3Bf (C fp32), kMmE2m1 (either).
hipError_t launch_mm_mx4(int fa, bool out_bf16, const MmParams& p, const Launch& s);
hipError_t launch_mm_f32_by_bf16(const MmParams& p, const Launch& s);
// bf16 NN into fp32 parts.
hipError_t launch_mm_bf16_parts(const MmParams& p, const Launch& s);

// How the backward divides its sums.  NN: tiles of 64 x 128 fewer than half the
// blocks that fit on the chip are multiplied by chunks of K, of 256 elements or
// more in multiples of 128, and what is left (0: whole).  TN: an expert's rows, experts being few, are added up
// in parts for one of two reasons (0: whole).  Tiles (128 x 128; 64 x 64 in fp32)
// that leave CUs without work: n parts, which save (1 - 1 / n) of an expert's
// rows at 10 ns each (20), and cost 8 bytes an element to write and read, 1.6 ps;
// three or more, as two save less than the launch that adds them up (E = 1, 768 x
// 2432, us with parts and without: 4096 rows 34 and 42, of 1024 25 and 15 in four
// parts; fp32 256 x 768, 4096 rows 27 and 73).  Experts with several times the
// others' rows: parts of five fourths of the average (us with and without, the
// largest expert in brackets, last where all have as many: 768 x 2432, E = 8, 4096
// rows on average (9000) 182 and 200, (16384) 150 and 322, 126 and 116; 2048 (4500)
// 104 and 105, 73 and 63; E = 16, 4096 (14000) 289 and 319, 259 and 245; 2048 (7000)
// 166 and 162, 142 and 125).  In fp32 this is for small matrices, of which an expert
// has fewer tiles than there are CUs, and costs up to an eighth in large ones (E =
// 8, 256 x 768, 1024 (2252) 43 and 65, (4096) 49 and 111, 46 and 42; 512 (1126) 28 and
// 36, 30 and 27; 768 x 768, 1024 (2252) 100 and 92, (4096) 103 and 125, 94 and 90; 768 x
// 2432, 1024 (2250) 261 and 241, 253 and 250; 512 (1100) 149 and 130, 143 and 132;
// 256 (540) 101 and 78, 93 and 79).
inline int mm_nn_chunk(int64_t R, int64_t N, int64_t K, int E) {
  const int64_t experts = E < R ? E : R;
  if (experts <= 0) return 0;
  const int64_t tiles = ((R + E - 1) / E + 63) / 64 * experts * ((N + 127) / 128);
  int64_t chunks = 512 / tiles;
  if (chunks > 16) chunks = 16;
  if (chunks > K / 256) chunks = K / 256;
  if (chunks < 2) return 0;
  return int(((K + chunks - 1) / chunks + 127) / 128 * 128);
}
inline int64_t mm_chunks(int64_t K, int kchunk) { return kchunk > 0 ? (K + kchunk - 1) / kchunk : 1; }
constexpr int kMmPartExperts = 64;  // lanes of a wavefront, which number the parts
inline int mm_tn_most(int64_t R, int64_t M, int64_t N, int E, bool f32) {
  const int64_t mean = R / E, side = f32 ? 64 : 128, gain = f32 ? 12800 : 6400;
  if (E > 16 || mean < 256) return 0;
  const int64_t tiles = (M + side - 1) / side * ((N + side - 1) / side) * E;
  int64_t parts = 1;
  while (parts < 512 / tiles && (parts + 1) * (parts + 1) * E * M * N <= mean * gain) ++parts;
  int64_t most = (mean + parts - 1) / parts;
  if (parts < 3) {
    if (E < 2 || (f32 ? mean < 500 : mean <= 2048)) return 0;
    most = mean * 5 / 4;
  }
  // (a gigabyte of parts at most)
  if (2 * (R / most) * M * N * 4 > int64_t(1) << 30) return 0;
  return int((most + 31) / 32 * 32);
}
// The parts kept: those of experts with more rows than `most`, of which there are
// R / most at most; each has one part more than its rows / most at most.
__host__ __device__ inline int64_t mm_tn_parts(int64_t R, int most, int E) {
  const int64_t n = most > 0 ? R / most : 0;
  return n + (n < E ? n : E);
}
// Units: an expert's parts, or its whole.
__host__ __device__ inline int64_t mm_tn_units(int64_t R, int most, int E) {
  return E + (most > 0 ? R / most : 0);
}
// Whether the experts with the longest sums start first; of short sums (E = 64,
// 48 rows each, fp32 768 x 256) finding them costs more than it saves: 50 against
// 32 us.
__host__ __device__ inline bool mm_tn_sorted(int64_t R, int E) {
  return E <= kMmPartExperts && R / E >= 256;
}
// NN: out [R, N] = the sum of the chunks, rounded once to the dtype.
hipError_t launch_mm_sum_chunks(const float* part, int64_t chunks, int64_t R, int64_t N, int dtype,
                                void* out, int64_t ldo, const Launch& s);
// TN: the experts of more than one part.
hipError_t launch_mm_sum_rows(const MmParams& p, int dtype, const Launch& s);

// ---- 4-bit values (mx4.hip): q [R, C / 2], scale [R, ceil(C / 32)], dense
hipError_t launch_mx4_pack(const void* x, int64_t ldx, int64_t R, int64_t C, int dtype, uint8_t* q,
                           uint8_t* scale, const Launch& s);
hipError_t launch_mx4_unpack(const uint8_t* q, const uint8_t* scale, int64_t R, int64_t C,
                             int dtype, void* x, int64_t ldx, const Launch& s);

}  // namespace topmoe
