// Products of grouped rows with matrices in 4 bits.
//
// By rows an expert (us; E = 8, 768 -> 4864 / E = 16, 2048 -> 1408 / E = 1, 2048 ->
// 6464).  The kernel for few rows, and 64 x 128:
//   bf16 rows   8: 9.5, 12.7 / 12.8, 22.1 / 5.9, 17.5;  16: 10.4, 12.9 / 16.5, 22.7 / 6.9,
//     17.5;  64: 27, 14.4 / 43, 24.8 / 14.6, 21.7
//   4-bit rows  8: 6.3, 9.9 / 10.9, 10.8 / 6.2, 8.5;  16: 7.3, 10.1 / 12.6, 11.0 / 6.2, 8.5;
//     64: 14.2, 11.3 / 29.9, 12.2 / 10.6, 9.3
//   8-bit rows  8: 6.6, 8.5 (2 rows) / 10.1, 14.1 / 6.1, 10.8;  16: 8.8, 8.9 / 13.7, 14.3 / 6.4,
//     10.9;  64: 18.2, 10.3 / 35.9, 16.3 / 12.1, 12.2
// 64 x 128, 128 x 256 and 256 x 256:
//   bf16 rows   256: 29.8, 28.2, 28.1 / 43.9, 38.8, 49.9 / 19.7, 34.4, 47;  512: 47.4, 40.3,
//     48.4 / 74, 63.8, 58.8 / 25.8, 35.4, 47.4;  2048: 177, 133, 132 / 278, 202, 206 / 75.5, 61.2,
//     56.2
//   4-bit rows  256: 20.4, 18, 19 / 25, 21.1, 24.3 / 9.9, 18.1, 21.8;  512: 29.5, 22.8, 29.9 /
//     37.8, 31.4, 27.1 / 15.1, 19.2, 22.7;  2048: 104, 76.7, 86.3 / 134, 97.5, 89.2 / 40.2, 31.4,
//     26.1 (of two blocks a CU with 128 x 256 one stores while the other
//     multiplies, which counts where K is short)
//   8-bit rows  256: 20.3, 21.2, 20.1 / 30.3, 24.3, 34.1 / 14.1, 21.1, 32.1;  512: 30.1, 29.5,
//     32.5 / 42.8, 41, 36.8 / 17.4, 22.1, 32.6;  2048: 109, 96.6, 87.4 / 159, 140, 126 / 44.3,
//     40.9, 36.3
#include "mm_few.h"

namespace topmoe {

namespace {

// The kernel for few rows: to 8 and 16 rows an expert, and to 32 where 64 x 128
// tiles are fewer than a quarter of the CUs.
template <int FA, int FB, typename OT>
bool few(const MmParams& p, const Launch& s, hipError_t* e) {
  using namespace mm;
  const int64_t rows = mm_rows_each(p);
  if (rows > 32 || (rows > 16 && mm_tiles(p, 64, 128) > 64)) return false;
  *e = rows <= 8 ? launch_few<FA, FB, OT, 1, 2, 8>(p, s) : launch_few<FA, FB, OT, 2, 2, 4>(p, s);
  return true;
}

// The scales of every row lie at multiples of four bytes: their rows are and
// they begin there.  Else all products that are not few rows' take 64 x 128 tiles
// with ordinary loads of the scales, which wait for all loads in flight (16384
// rows, us: K = 2080 for 2048, to 6464: 422 for 147 of 4-bit rows, 441 for 211 of
// 8-bit, 739 for 380 of bf16; K = 6464 for 6400, to 2048: 673 for 141, 691 for 168,
// 1039 for 322).
bool words(const MmParams& p) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.As) | reinterpret_cast<uintptr_t>(p.Bs);
  return p.K % 128 == 0 && at % 4 == 0;
}
template <int FA, int FB, typename OT, int Q, int S>
hipError_t small(const MmParams& p, const Launch& s) {
  using namespace mm;
  return words(p) ? launch_tile<kMmNT, FA, FB, OT, 64, 128, 2, 2, Q, S, true>(p, s)
                  : launch_tile<kMmNT, FA, FB, OT, 64, 128, 2, 2, Q, S, false>(p, s);
}

}  // namespace

hipError_t launch_mm_mx4(int fa, bool out_bf16, const MmParams& p, const Launch& s) {
  using namespace mm;
  hipError_t e = hipSuccess;
  const bool large = words(p) && mm_tiles(p, 256, 256) >= 140;
  const bool mid = words(p) && mm_tiles(p, 128, 256) >= 140;
  switch (fa) {
    case kMmBf16:
      if (few<kMmBf16, kMmE2m1Bf, bf16_t>(p, s, &e)) return e;
      if (large)
        return launch_tile<kMmNT, kMmBf16, kMmE2m1Bf, bf16_t, 256, 256, 2, 4, 4, 3>(p, s);
      if (mid) return launch_tile<kMmNT, kMmBf16, kMmE2m1Bf, bf16_t, 128, 256, 2, 2, 4, 3>(p, s);
      return small<kMmBf16, kMmE2m1Bf, bf16_t, 4, 4>(p, s);
    case kMmF32Split:
      if (few<kMmF32Split, kMmE2m1Bf, float>(p, s, &e)) return e;
      return small<kMmF32Split, kMmE2m1Bf, float, 4, 3>(p, s);
    case kMmE4m3:
      if (few<kMmE4m3, kMmE2m1, bf16_t>(p, s, &e)) return e;
      if (large) return launch_tile<kMmNT, kMmE4m3, kMmE2m1, bf16_t, 256, 256, 4, 2, 2, 3>(p, s);
      if (mid) return launch_tile<kMmNT, kMmE4m3, kMmE2m1, bf16_t, 128, 256, 2, 4, 2, 3>(p, s);
      return small<kMmE4m3, kMmE2m1, bf16_t, 2, 3>(p, s);
    case kMmE4m3Bf:
      if (few<kMmE4m3Bf, kMmE2m1Bf, float>(p, s, &e)) return e;
      return small<kMmE4m3Bf, kMmE2m1Bf, float, 4, 3>(p, s);
    case kMmE2m1:
      if (!out_bf16) {
        if (few<kMmE2m1, kMmE2m1, float>(p, s, &e)) return e;
        return small<kMmE2m1, kMmE2m1, float, 2, 4>(p, s);
      }
      if (few<kMmE2m1, kMmE2m1, bf16_t>(p, s, &e)) return e;
      if (large && p.K >= 1024)
        return launch_tile<kMmNT, kMmE2m1, kMmE2m1, bf16_t, 256, 256, 2, 4, 2, 4>(p, s);
      if (mid) return launch_tile<kMmNT, kMmE2m1, kMmE2m1, bf16_t, 128, 256, 2, 2, 2, 3>(p, s);
      return small<kMmE2m1, kMmE2m1, bf16_t, 2, 4>(p, s);
  }
  return hipErrorInvalidValue;
}

// dx = dy W with dy in fp32 and W in bf16.  (E = 4, 2432 -> 768, 258 rows each: three
// slots 47 us, four 49; 2048 rows each 120 and 136.)
hipError_t launch_mm_f32_by_bf16(const MmParams& p, const Launch& s) {
  return mm::launch_tile<kMmNN, kMmF32Split, kMmBf16, float, 64, 128, 2, 2, 2, 3>(p, s);
}

}  // namespace topmoe
