// Values in 8 bits: a thread's channels to and from e4m3 with their group's
// scale byte (the format is described in act8.hip), and SiLU of them.
#pragma once

#include "device_common.h"

namespace topmoe {

// E channels a thread, 32 / E lanes a group.
template <int E>
constexpr int kGroupLanes = 32 / E;

// Largest over the four or eight lanes of a group, in each of them.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  static_assert(LANES == 4 || LANES == 8, "lanes of a group");
  uint32_t w = uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0xB1, 0xF, 0xF, false));  // lane ^ 1
  v = v > w ? v : w;
  w = uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x4E, 0xF, 0xF, false));  // lane ^ 2
  v = v > w ? v : w;
  if constexpr (LANES == 8) {  // row_half_mirror: the other quad of the eight
    w = uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x141, 0xF, 0xF, false));
    v = v > w ? v : w;
  }
  return v;
}

// E channels of a group to E bytes (in words) and the group's scale byte.
// Every lane of the group must take part (lanes past the row's end with zeros).
// Magnitudes are compared as their fp32 bits, which are ordered like them.
template <int E>
__device__ __forceinline__ uint32_t pack_q(const float (&x)[E], uint32_t (&q)[E / 4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
    m = b < 0x7f800000u && b > m ? b : m;
  }
  m = group_max<kGroupLanes<E>>(m);
  // 448 = 1.75 * 2^8: the exponent less 8, one more for a fraction above 1.75
  int e = int(m >> 23) - 135 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < -127 ? -127 : e;
  const float inv = __uint_as_float(uint32_t(127 - e) << 23);  // 2^-e, e in [-127, 120]
  float v[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const bool fine = (__float_as_uint(x[i]) & 0x7fffffffu) < 0x7f800000u;
    v[i] = fine ? x[i] * inv : __uint_as_float(0x7fc00000u);
  }
#pragma unroll
  for (int w = 0; w < E / 4; ++w) {
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

template <int E>
__device__ __forceinline__ void unpack_q(const uint32_t (&q)[E / 4], float s, float (&v)[E]) {
#pragma unroll
  for (int w = 0; w < E / 4; ++w) {
    v[4 * w + 0] = __builtin_amdgcn_cvt_f32_fp8(int(q[w]), 0) * s;
    v[4 * w + 1] = __builtin_amdgcn_cvt_f32_fp8(int(q[w]), 1) * s;
    v[4 * w + 2] = __builtin_amdgcn_cvt_f32_fp8(int(q[w]), 2) * s;
    v[4 * w + 3] = __builtin_amdgcn_cvt_f32_fp8(int(q[w]), 3) * s;
  }
}

__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.4426950408889634f));
}
// SiLU(g) first: g * u may pass fp32's range where SiLU(g) * u does not.
__device__ __forceinline__ float silu(float g) { return g * sigmoid(g); }

}  // namespace topmoe
