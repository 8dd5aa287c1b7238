// Products of grouped rows with matrices in 4 bits.
//
// By rows an expert (us; E = 8, 768 -> 4864 / E = 16, 2048 -> 1408 / E = 1, 2048 ->
// 6464), the kernel for few rows, 64 x 128 and large tiles:
//   bf16 rows   8: 9.5, 12.7, - / 12.8, 22.1, - / 5.9, 17.5, -;  16: 10.4, 12.9 / 16.5,
//     22.7 / 6.9, 17.5;  64: 27, 14.4 / 43, 24.8 / 14.6, 21.7;  2048: -, 169, 127 / -, 251,
//     208 / -, 76.6, 61.1
//   4-bit rows  8: 6.3, 9.9 / 10.9, 10.8 / 6.2, 8.5;  16: 7.3, 10.1 / 12.6, 11.0 / 6.2, 8.5;
//     64: 14.2, 11.3 / 29.9, 12.2 / 10.6, 9.3;  2048: -, 121, 95 / -, 118, 97.5 / -, 38.6, 27.7
//   8-bit rows  8: 6.6, 8.5 (2 rows) / 10.1, 14.1 / 6.1, 10.8;  16: 8.8, 8.9 / 13.7, 14.3 / 6.4,
//     10.9;  64: 18.2, 10.3 / 35.9, 16.3 / 12.1, 12.2;  2048: -, 116, 93 / -, 170, 144 / -, 51, 42
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

}  // namespace

hipError_t launch_mm_mx4(int fa, bool out_bf16, const MmParams& p, const Launch& s) {
  using namespace mm;
  hipError_t e = hipSuccess;
  switch (fa) {
    case kMmBf16:
      if (few<kMmBf16, kMmE2m1Bf, bf16_t>(p, s, &e)) return e;
      if (mm_tiles(p, 256, 256) >= 140)
        return launch_tile<kMmNT, kMmBf16, kMmE2m1Bf, bf16_t, 256, 256, 2, 4, 4, 3>(p, s);
      return launch_tile<kMmNT, kMmBf16, kMmE2m1Bf, bf16_t, 64, 128, 2, 2, 4, 4>(p, s);
    case kMmF32Split:
      if (few<kMmF32Split, kMmE2m1Bf, float>(p, s, &e)) return e;
      return launch_tile<kMmNT, kMmF32Split, kMmE2m1Bf, float, 64, 128, 2, 2, 4, 3>(p, s);
    case kMmE4m3:
      if (few<kMmE4m3, kMmE2m1, bf16_t>(p, s, &e)) return e;
      if (mm_tiles(p, 128, 256) >= 200)
        return launch_tile<kMmNT, kMmE4m3, kMmE2m1, bf16_t, 128, 256, 2, 4, 2, 3>(p, s);
      return launch_tile<kMmNT, kMmE4m3, kMmE2m1, bf16_t, 64, 128, 2, 2, 2, 3>(p, s);
    case kMmE4m3Bf:
      if (few<kMmE4m3Bf, kMmE2m1Bf, float>(p, s, &e)) return e;
      return launch_tile<kMmNT, kMmE4m3Bf, kMmE2m1Bf, float, 64, 128, 2, 2, 4, 3>(p, s);
    case kMmE2m1:
      if (!out_bf16) {
        if (few<kMmE2m1, kMmE2m1, float>(p, s, &e)) return e;
        return launch_tile<kMmNT, kMmE2m1, kMmE2m1, float, 64, 128, 2, 2, 2, 4>(p, s);
      }
      if (few<kMmE2m1, kMmE2m1, bf16_t>(p, s, &e)) return e;
      if (mm_tiles(p, 256, 256) >= 200)
        return launch_tile<kMmNT, kMmE2m1, kMmE2m1, bf16_t, 256, 256, 4, 2, 2, 4>(p, s);
      return launch_tile<kMmNT, kMmE2m1, kMmE2m1, bf16_t, 64, 128, 2, 2, 2, 4>(p, s);
  }
  return hipErrorInvalidValue;
}

// dx = dy W with dy in fp32 and W in bf16.
hipError_t launch_mm_f32_by_bf16(const MmParams& p, const Launch& s) {
  return mm::launch_tile<kMmNN, kMmF32Split, kMmBf16, float, 64, 128, 2, 2, 2, 4>(p, s);
}

}  // namespace topmoe
