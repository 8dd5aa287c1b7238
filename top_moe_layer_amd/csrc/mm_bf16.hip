// bf16 products of grouped rows: y = x W^T, dx = dy W, dW = dy^T x.
#include "mm_few.h"

namespace topmoe {

hipError_t launch_mm_bf16(MmLayout layout, const MmParams& p, const Launch& s) {
  using namespace mm;
  switch (layout) {
    case kMmNT:
      if (mm_few(p, 32)) {
        if (mm_rows_each(p) <= 16) return launch_few<kMmBf16, kMmBf16, bf16_t, 1, 2, 8>(p, s);
        return launch_few<kMmBf16, kMmBf16, bf16_t, 2, 2, 8>(p, s);
      }
      if (mm_rows_each(p) <= 512) return launch_tile<kMmNT, kMmBf16, kMmBf16, bf16_t, 128, 128, 2, 2, 3>(p, s);
      return launch_tile<kMmNT, kMmBf16, kMmBf16, bf16_t, 256, 256, 2, 4, 2>(p, s);
    case kMmNN:
      if (mm_rows_each(p) <= 512) return launch_tile<kMmNN, kMmBf16, kMmBf16, bf16_t, 128, 128, 2, 2, 3>(p, s);
      return launch_tile<kMmNN, kMmBf16, kMmBf16, bf16_t, 256, 256, 2, 4, 2>(p, s);
    case kMmTN:
      return launch_tile<kMmTN, kMmBf16, kMmBf16, bf16_t, 128, 128, 2, 2, 3>(p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace topmoe
