// bf16 products of grouped rows: y = x W^T, dx = dy W, dW = dy^T x.
//
// Shapes by the tiles they make for 256 CUs (us; rows an expert -> time):
//   y, 64 x 64, 128 x 256, 256 x 256: E = 8, 768 -> 4864  64: 16.9, 19, 19.4; 256:
//     33.6, 32.1, 28.2; 512: 69.3, 51.3, 56; 2048: 219, 159, 157;  E = 16, 2048 -> 1408  64:
//     26.2, 42.4, 42.2; 256: 56, 49.4, 58.2; 512: 101, 76.2, 64.3; 2048: 324, 251, 233;  E = 1,
//     2048 -> 6464  256: 15.5, 35.6, 43.1; 1024: 42, 40.3, 45.4; 2048: 77.1, 68.9, 54.5
//   64 x 128 and 64 x 64: E = 8, 64 rows 15.6 and 17.2; E = 16, 32 rows 23 and 20.8,
//     128 rows 32.5 and 39.2; E = 1, 128 rows 16.6 and 10.6
//   dx of the same, 64 x 128, 128 x 256, 256 x 256 (E = 8, E = 16):  256: 32.3, 73.8,
//     99.7, 58.9, 53.7, 45.3; 1024: 128, 97.5, 124, 176, 127, 125; 2048: 219, 148, 135, 314, 218, 220
//   dW, 128 x 128, 128 x 256, 256 x 256, rows an expert all alike: E = 8, 768 x 2432
//     64: 15.6, 11.2, 12.7; 512: 27.9, 24.3, 23.7; 4096: 141, 124, 125;  E = 16, 2048 x 1408,
//     1024: 122, 106, 107;  E = 64, 768 x 2432, 512: 258, 215, 224;  E = 4, 1024: 23.5, 25.8,
//     35.2;  E = 1, 1024: 14.6, 21, 28.7
// The kernel for few rows, whose wavefronts divide K, where even 64 x 64 tiles
// leave CUs without work (E = 1, 2 rows: 7.5 against 9.2; E = 16, 8 rows, 352
// tiles: 21.2 against 19.0).
#include "mm_few.h"

namespace topmoe {

hipError_t launch_mm_bf16(MmLayout layout, const MmParams& p, const Launch& s) {
  using namespace mm;
  const bool large = mm_tiles(p, 256, 256) >= 140, mid = mm_tiles(p, 128, 256) >= 140;
  switch (layout) {
    case kMmNT:
      if (mm_rows_each(p) <= 16 && mm_tiles(p, 64, 64) <= 256)
        return launch_few<kMmBf16, kMmBf16, bf16_t, 1, 2, 8>(p, s);
      if (large) return launch_tile<kMmNT, kMmBf16, kMmBf16, bf16_t, 256, 256, 2, 4, 2, 4>(p, s);
      if (mid) return launch_tile<kMmNT, kMmBf16, kMmBf16, bf16_t, 128, 256, 2, 2, 2, 3>(p, s);
      if (mm_tiles(p, 64, 128) >= 256)
        return launch_tile<kMmNT, kMmBf16, kMmBf16, bf16_t, 64, 128, 2, 2, 4, 3>(p, s);
      return launch_tile<kMmNT, kMmBf16, kMmBf16, bf16_t, 64, 64, 2, 2, 4, 4>(p, s);
    case kMmNN:
      if (large) return launch_tile<kMmNN, kMmBf16, kMmBf16, bf16_t, 256, 256, 2, 4, 2, 4>(p, s);
      if (mid) return launch_tile<kMmNN, kMmBf16, kMmBf16, bf16_t, 128, 256, 2, 2, 2, 3>(p, s);
      return launch_tile<kMmNN, kMmBf16, kMmBf16, bf16_t, 64, 128, 2, 2, 4, 3>(p, s);
    case kMmTN: {
      const int64_t sums = p.most > 0 && p.R / p.most > p.E ? p.R / p.most : p.E;
      if (mm_tn_tiles(p, 256, 256) * sums >= 200 && p.R / p.E >= 1024)
        return launch_tile<kMmTN, kMmBf16, kMmBf16, bf16_t, 256, 256, 2, 4, 2, 4>(p, s);
      if (mm_tn_tiles(p, 128, 256) * sums >= 256)
        return launch_tile<kMmTN, kMmBf16, kMmBf16, bf16_t, 128, 256, 2, 2, 2, 3>(p, s);
      return launch_tile<kMmTN, kMmBf16, kMmBf16, bf16_t, 128, 128, 2, 2, 2, 4>(p, s);
    }
  }
  return hipErrorInvalidValue;
}

hipError_t launch_mm_bf16_parts(const MmParams& p, const Launch& s) {
  return mm::launch_tile<kMmNN, kMmBf16, kMmBf16, float, 64, 128, 2, 2, 4, 3>(p, s);
}

}  // namespace topmoe
