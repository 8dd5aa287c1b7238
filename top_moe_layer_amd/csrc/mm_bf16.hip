// bf16 products of grouped rows: y = x W^T, dx = dy W, dW = dy^T x.
//
// Shapes by the tiles they make for 256 CUs (us; rows an expert -> time):
//   E = 8, 768 -> 4864   128 rows: 64 x 64 19.7, 128 x 256 21.4, 256 x 256 23.5;
//     256: 33.4, 33.2, 30.1; 2048: 212, 164, 158
//   E = 16, 2048 -> 1408   32: 21.3, 39.1, 43.5; 256: 55.4, 48.1, 58.6; 2048: 321, 254, 237
//   E = 1, 2048 -> 6464  256: 15.3, 35.0, 45.2; 1024: 43.1, 38.8, 50.4; 2048: 77.6, 69.6, 61.5
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
      return launch_tile<kMmNT, kMmBf16, kMmBf16, bf16_t, 64, 64, 2, 2, 4, 4>(p, s);
    case kMmNN:
      if (large) return launch_tile<kMmNN, kMmBf16, kMmBf16, bf16_t, 256, 256, 2, 4, 2, 4>(p, s);
      if (mid) return launch_tile<kMmNN, kMmBf16, kMmBf16, bf16_t, 128, 256, 2, 2, 2, 3>(p, s);
      return launch_tile<kMmNN, kMmBf16, kMmBf16, bf16_t, 64, 128, 2, 2, 2, 4>(p, s);
    case kMmTN:
      return launch_tile<kMmTN, kMmBf16, kMmBf16, bf16_t, 128, 256, 2, 2, 2, 3>(p, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_mm_bf16_parts(const MmParams& p, const Launch& s) {
  return mm::launch_tile<kMmNN, kMmBf16, kMmBf16, float, 64, 128, 2, 2, 2, 4>(p, s);
}

}  // namespace topmoe
