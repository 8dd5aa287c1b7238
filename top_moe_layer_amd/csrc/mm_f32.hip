// fp32 products of grouped rows: y = x W^T, dx = dy W, dW = dy^T x.
#include "mm_few.h"

namespace topmoe {

hipError_t launch_mm_f32(MmLayout layout, const MmParams& p, const Launch& s) {
  using namespace mm;
  switch (layout) {
    case kMmNT:
      if (mm_few(p, 32)) {
        if (mm_rows_each(p) <= 16) return launch_few<kMmF32, kMmF32, float, 1, 2, 8>(p, s);
        return launch_few<kMmF32, kMmF32, float, 2, 2, 8>(p, s);
      }
      return launch_tile<kMmNT, kMmF32, kMmF32, float, 128, 128, 2, 2, 3>(p, s);
    case kMmNN:
      return launch_tile<kMmNN, kMmF32, kMmF32, float, 128, 128, 2, 2, 3>(p, s);
    case kMmTN:
      return launch_tile<kMmTN, kMmF32, kMmF32, float, 128, 128, 2, 2, 3>(p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace topmoe
