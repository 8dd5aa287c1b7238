// Values in 8 bits: eight channels to and from e4m3 with their group's scale
// byte (the format is described in act8.hip).
#pragma once

#include "device_common.h"

namespace topmoe {

// Largest magnitude over the four lanes of a quad, as its fp32 bits (ordered
// like the magnitudes).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t w = uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0xB1, 0xF, 0xF, false));  // lane ^ 1
  v = v > w ? v : w;
  w = uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x4E, 0xF, 0xF, false));  // lane ^ 2
  return v > w ? v : w;
}

// Eight channels of a group to 8 bytes and the group's scale byte.  Every lane
// of the quad must take part (lanes past the row's end with zeros).
__device__ __forceinline__ uint32_t pack8(const float (&x)[8], uint32_t (&q)[2]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
    m = b < 0x7f800000u && b > m ? b : m;
  }
  m = quad_max(m);
  // 448 = 1.75 * 2^8: the exponent less 8, one more for a fraction above 1.75
  int e = int(m >> 23) - 135 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < -127 ? -127 : e;
  const float inv = __uint_as_float(uint32_t(127 - e) << 23);  // 2^-e, e in [-127, 120]
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool fine = (__float_as_uint(x[i]) & 0x7fffffffu) < 0x7f800000u;
    v[i] = fine ? x[i] * inv : __uint_as_float(0x7fc00000u);
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    int d = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * w], v[4 * w + 1], 0, false);
    q[w] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * w + 2], v[4 * w + 3], d, true));
  }
  return uint32_t(e + 127);
}

// 2^(byte - 127) (a byte of 0 is the subnormal 2^-127; 255 is NaN).
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte == 0 ? __uint_as_float(0x00400000u)
                   : byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ void unpack_q8(const uint32_t (&q)[2], float s, float (&v)[8]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    v[4 * w + 0] = __builtin_amdgcn_cvt_f32_fp8(int(q[w]), 0) * s;
    v[4 * w + 1] = __builtin_amdgcn_cvt_f32_fp8(int(q[w]), 1) * s;
    v[4 * w + 2] = __builtin_amdgcn_cvt_f32_fp8(int(q[w]), 2) * s;
    v[4 * w + 3] = __builtin_amdgcn_cvt_f32_fp8(int(q[w]), 3) * s;
  }
}

}  // namespace topmoe
