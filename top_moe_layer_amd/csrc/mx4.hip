// Values in 4 bits: OCP microscaling e2m1 (fp4).
//
// Each group of 32 consecutive channels of a row (the row's last group may be
// shorter) shares one power-of-two scale 2^e and stores its elements as e2m1
// values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) of x * 2^-e, rounded
// to nearest, ties to the even code: e is the smallest integer (at least -127)
// for which the group's largest magnitude is at most 6 * 2^e, so nothing
// saturates, and the scaling itself is exact.  The scale is stored as the byte
// e + 127; two elements share a byte, the first in its low half.  e2m1 has no
// infinity or NaN: a group with an element that is not finite has the scale
// byte 255, OCP's NaN, and all of it reads back as NaN.
//
// A thread converts 16 bytes of a row (8 bf16 or 4 fp32 channels) in registers
// with v_cvt_scalef32_pk_fp4_f32; the four or eight threads of a group find its
// largest magnitude with two or three lane exchanges.  Bound by memory: 16 x 2432
// x 2048 bf16 packed in 36 us and unpacked in 29 (202 MB each, 5.5 and 6.9 TB/s).
#include "act8_impl.h"
#include "mm.h"

#include "../../include/topmoe.h"

namespace topmoe {

namespace {

// Largest over a group of the bits of the magnitudes: infinities and NaN are above the rest.
template <int E>
__device__ __forceinline__ uint32_t pack4(const float (&x)[E], uint32_t& q) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  m = group_max<kGroupLanes<E>>(m);
  q = 0;
  if (m >= 0x7f800000u) return 255u;
  // 6 = 1.5 * 2^2: the exponent less 2, one more for a fraction above 1.5
  int e = int(m >> 23) - 129 + ((m & 0x7fffffu) > 0x400000u ? 1 : 0);
  e = e < -127 ? -127 : e;
  const float s = e == -127 ? __uint_as_float(0x00400000u) : __uint_as_float(uint32_t(e + 127) << 23);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[0], x[1], s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[2], x[3], s, 1);
  if constexpr (E == 8) {
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[4], x[5], s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[6], x[7], s, 3);
  }
  return uint32_t(e + 127);
}

// Through bf16, which holds every e2m1 value times a scale exactly but for
// 4 * 2^126 and more, infinite in fp32 as well.
template <int SEL>
__device__ __forceinline__ void unpack4(uint32_t q, float s, float& a, float& b) {
  const uint32_t w =
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, SEL));
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}

template <typename T>
__global__ __launch_bounds__(256) void mx4_pack_kernel(const T* __restrict__ x, int64_t ldx,
                                                       int64_t r0, uint32_t pieces, uint32_t pp,
                                                       int C, uint8_t* __restrict__ q,
                                                       uint8_t* __restrict__ scale) {
  const Place<T> a(r0, pieces, pp, C);
  constexpr int E = kE<T>;
  float v[E];
  unpack(load_piece_if<true>(a.in, x + a.at(ldx)), v);
  uint32_t b;
  const uint32_t s = pack4<E>(v, b);
  if (a.in) {
    uint8_t* o = q + a.at(C) / 2;
    if constexpr (E == 8) *reinterpret_cast<uint32_t*>(o) = b;
    else *reinterpret_cast<uint16_t*>(o) = uint16_t(b);
  }
  if (a.first()) scale[a.group()] = uint8_t(s);
}

template <typename T, bool NT>
__global__ __launch_bounds__(256) void mx4_unpack_kernel(const uint8_t* __restrict__ q,
                                                         const uint8_t* __restrict__ scale,
                                                         int64_t r0, uint32_t pieces, uint32_t pp,
                                                         int C, T* __restrict__ x, int64_t ldx) {
  const Place<T> a(r0, pieces, pp, C);
  constexpr int E = kE<T>;
  if (!a.in) return;
  const uint8_t* at = q + a.at(C) / 2;
  uint32_t b;
  if constexpr (E == 8) b = *reinterpret_cast<const uint32_t*>(at);
  else b = *reinterpret_cast<const uint16_t*>(at);
  const float s = scale_of(scale[a.group()]);
  float v[E];
  unpack4<0>(b, s, v[0], v[1]);
  unpack4<1>(b, s, v[2], v[3]);
  if constexpr (E == 8) {
    unpack4<2>(b, s, v[4], v[5]);
    unpack4<3>(b, s, v[6], v[7]);
  }
  store_piece<NT>(x + a.at(ldx), v);
}

template <typename T>
hipError_t pack_typed(const void* x, int64_t ldx, int64_t R, int64_t C, uint8_t* q, uint8_t* scale,
                      const Launch& s) {
  return for_slabs<T>(R, C, s, [&](dim3 grid, int64_t r0, uint32_t pieces, uint32_t pp,
                                   const Launch& L) {
    return launch_kernel(mx4_pack_kernel<T>, grid, dim3(256), 0, L, static_cast<const T*>(x), ldx,
                         r0, pieces, pp, int(C), q, scale);
  });
}

template <typename T, bool NT>
hipError_t unpack_typed(const uint8_t* q, const uint8_t* scale, int64_t R, int64_t C, void* x,
                        int64_t ldx, const Launch& s) {
  return for_slabs<T>(R, C, s, [&](dim3 grid, int64_t r0, uint32_t pieces, uint32_t pp,
                                   const Launch& L) {
    return launch_kernel(mx4_unpack_kernel<T, NT>, grid, dim3(256), 0, L, q, scale, r0, pieces, pp,
                         int(C), static_cast<T*>(x), ldx);
  });
}

}  // namespace

hipError_t launch_mx4_pack(const void* x, int64_t ldx, int64_t R, int64_t C, int dtype, uint8_t* q,
                           uint8_t* scale, const Launch& s) {
  return dtype == TOPMOE_DTYPE_FP32 ? pack_typed<float>(x, ldx, R, C, q, scale, s)
                                    : pack_typed<bf16_t>(x, ldx, R, C, q, scale, s);
}

hipError_t launch_mx4_unpack(const uint8_t* q, const uint8_t* scale, int64_t R, int64_t C,
                             int dtype, void* x, int64_t ldx, const Launch& s) {
  if (dtype == TOPMOE_DTYPE_FP32)
    return R * C * 4 >= kNtBytes ? unpack_typed<float, true>(q, scale, R, C, x, ldx, s)
                                 : unpack_typed<float, false>(q, scale, R, C, x, ldx, s);
  return R * C * 2 >= kNtBytes ? unpack_typed<bf16_t, true>(q, scale, R, C, x, ldx, s)
                               : unpack_typed<bf16_t, false>(q, scale, R, C, x, ldx, s);
}

}  // namespace topmoe
