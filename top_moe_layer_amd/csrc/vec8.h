// Eight consecutive values of the dtype (16 bytes of bf16, 32 of fp32), the
// unit the row-wise kernels move: kept as loaded until used, so that rows held
// in registers cost what they cost in memory.
#pragma once

#include "device_common.h"

namespace topmoe {

template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  u32x4 q;
};
template <>
struct Raw8<float> {
  f32x4 lo, hi;
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p);
template <>
__device__ __forceinline__ Raw8<bf16_t> load_raw8<bf16_t>(const bf16_t* p) {
  return Raw8<bf16_t>{*reinterpret_cast<const u32x4*>(p)};
}
template <>
__device__ __forceinline__ Raw8<float> load_raw8<float>(const float* p) {
  return Raw8<float>{*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)};
}

template <typename T>
__device__ __forceinline__ void store_raw8(T* p, const Raw8<T>& r);
template <>
__device__ __forceinline__ void store_raw8<bf16_t>(bf16_t* p, const Raw8<bf16_t>& r) {
  *reinterpret_cast<u32x4*>(p) = r.q;
}
template <>
__device__ __forceinline__ void store_raw8<float>(float* p, const Raw8<float>& r) {
  *reinterpret_cast<f32x4*>(p) = r.lo;
  *reinterpret_cast<f32x4*>(p + 4) = r.hi;
}

template <typename T>
__device__ __forceinline__ Raw8<T> zero_raw8();
template <>
__device__ __forceinline__ Raw8<bf16_t> zero_raw8<bf16_t>() {
  return Raw8<bf16_t>{u32x4{0u, 0u, 0u, 0u}};
}
template <>
__device__ __forceinline__ Raw8<float> zero_raw8<float>() {
  return Raw8<float>{f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
}

__device__ __forceinline__ void unpack8(const Raw8<bf16_t>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.q[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.q[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = r.lo[i];
    v[4 + i] = r.hi[i];
  }
}

// Rounded once to the dtype (nearest even).
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<bf16_t>(bf16_t* p, const float (&v)[8]) {
  u32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = uint32_t(f32_to_bf16(v[2 * i])) | (uint32_t(f32_to_bf16(v[2 * i + 1])) << 16);
  *reinterpret_cast<u32x4*>(p) = q;
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}

}  // namespace topmoe
