// fp32 products of grouped rows: y = x W^T, dx = dy W, dW = dy^T x.
//
// On the fp32 matrix instructions, a sixteenth of the bf16 rate, small tiles
// lose nothing: 64 x 64 against 128 x 128, E = 4, 768 -> 2432, 1024 rows each: y
// 133 against 148 us, dx 167 and 157, dW 136 and 145; 48 rows each: 17.8 and
// 49.8, 43 and 153, 19 and 24.  Few rows: E = 64, 768 -> 256, 4 rows each 13.3
// against 18.1 us, 16 each 17.3 and 18.1.  dW with three slots, which lets more
// blocks share a CU, against four: E = 64, 768 x 256, 48 rows each, which is the
// way of a block from its offsets to its stores, 31 and 35; E = 4, 768 x 2432,
// 1024 rows each 139 and 148.
#include "mm_few.h"

namespace topmoe {

hipError_t launch_mm_f32(MmLayout layout, const MmParams& p, const Launch& s) {
  using namespace mm;
  switch (layout) {
    case kMmNT:
      if (mm_rows_each(p) <= 8) return launch_few<kMmF32, kMmF32, float, 1, 2, 8>(p, s);
      if (mm_rows_each(p) <= 16) return launch_few<kMmF32, kMmF32, float, 2, 2, 8>(p, s);
      return launch_tile<kMmNT, kMmF32, kMmF32, float, 64, 64, 2, 2, 4, 4>(p, s);
    case kMmNN:
      return launch_tile<kMmNN, kMmF32, kMmF32, float, 64, 64, 2, 2, 4, 4>(p, s);
    case kMmTN:
      return launch_tile<kMmTN, kMmF32, kMmF32, float, 64, 64, 2, 2, 2, 3>(p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace topmoe
