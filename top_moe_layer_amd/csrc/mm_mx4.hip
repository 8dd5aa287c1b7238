// Products of grouped rows with matrices in 4 bits.
#include "mm_few.h"

namespace topmoe {

namespace {

template <int FA, int FB, typename OT, int BM, int BN, int WM, int WN, int S>
hipError_t run(const MmParams& p, const Launch& s) {
  using namespace mm;
  if (mm_few(p, 64)) {
    const int64_t rows = mm_rows_each(p);
    if (rows <= 16) return launch_few<FA, FB, OT, 1, 2, 8>(p, s);
    return launch_few<FA, FB, OT, 2, 2, 8>(p, s);
  }
  return launch_tile<kMmNT, FA, FB, OT, BM, BN, WM, WN, S>(p, s);
}

}  // namespace

hipError_t launch_mm_mx4(int fa, bool out_bf16, const MmParams& p, const Launch& s) {
  switch (fa) {
    case kMmBf16:
      return run<kMmBf16, kMmE2m1Bf, bf16_t, 256, 256, 2, 4, 3>(p, s);
    case kMmF32Split:
      return run<kMmF32Split, kMmE2m1Bf, float, 128, 128, 2, 2, 3>(p, s);
    case kMmE4m3:
      return run<kMmE4m3, kMmE2m1, bf16_t, 128, 128, 2, 2, 3>(p, s);
    case kMmE4m3Bf:
      return run<kMmE4m3Bf, kMmE2m1Bf, float, 128, 128, 2, 2, 3>(p, s);
    case kMmE2m1:
      return out_bf16 ? run<kMmE2m1, kMmE2m1, bf16_t, 128, 128, 2, 2, 3>(p, s)
                      : run<kMmE2m1, kMmE2m1, float, 128, 128, 2, 2, 3>(p, s);
  }
  return hipErrorInvalidValue;
}

// dx = dy W with dy in fp32 and W in bf16.
hipError_t launch_mm_f32_by_bf16(const MmParams& p, const Launch& s) {
  return mm::launch_tile<kMmNN, kMmF32Split, kMmBf16, float, 128, 128, 2, 2, 3>(p, s);
}

}  // namespace topmoe
