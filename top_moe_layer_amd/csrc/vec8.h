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

// 16 bytes to / from memory; NT: non-temporal, for data that this kernel reads
// or writes once and that nothing reads again while it is still in the caches.
template <bool NT, typename V>
__device__ __forceinline__ V load_vec(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load(static_cast<const V*>(p));
  return *static_cast<const V*>(p);
}
template <bool NT, typename V>
__device__ __forceinline__ void store_vec(void* p, V v) {
  if constexpr (NT) __builtin_nontemporal_store(v, static_cast<V*>(p));
  else *static_cast<V*>(p) = v;
}

template <typename T, bool NT = false>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p) {
  if constexpr (sizeof(T) == 2) return Raw8<T>{load_vec<NT, u32x4>(p)};
  else return Raw8<T>{load_vec<NT, f32x4>(p), load_vec<NT, f32x4>(p + 4)};
}

template <typename T, bool NT = false>
__device__ __forceinline__ void store_raw8(T* p, const Raw8<T>& r) {
  if constexpr (sizeof(T) == 2) {
    store_vec<NT, u32x4>(p, r.q);
  } else {
    store_vec<NT, f32x4>(p, r.lo);
    store_vec<NT, f32x4>(p + 4, r.hi);
  }
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
template <typename T, bool NT = false>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = uint32_t(f32_to_bf16(v[2 * i])) | (uint32_t(f32_to_bf16(v[2 * i + 1])) << 16);
    store_vec<NT, u32x4>(p, q);
  } else {
    store_vec<NT, f32x4>(p, f32x4{v[0], v[1], v[2], v[3]});
    store_vec<NT, f32x4>(p + 4, f32x4{v[4], v[5], v[6], v[7]});
  }
}

}  // namespace topmoe
