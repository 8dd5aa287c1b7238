// 16 bytes of a row (8 bf16 or 4 fp32 values), the piece a thread of the
// row-wise kernels moves at a time: consecutive lanes hold consecutive pieces,
// and a piece is kept as loaded until used, so that rows held in registers
// cost what they cost in memory.
#pragma once

#include "device_common.h"

namespace topmoe {

// Values in a piece.
template <typename T>
constexpr int kE = 16 / int(sizeof(T));

// A vector to / from memory; NT: non-temporal, for data that this kernel reads
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

template <bool NT = false>
__device__ __forceinline__ u32x4 load_piece(const void* p) {
  return load_vec<NT, u32x4>(p);
}
// Zeros where there is nothing to load.
template <bool NT = false>
__device__ __forceinline__ u32x4 load_piece_if(bool in, const void* p) {
  return in ? load_vec<NT, u32x4>(p) : u32x4{0u, 0u, 0u, 0u};
}

__device__ __forceinline__ void unpack(u32x4 q, float (&v)[8]) {  // bf16
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(q[i] << 16);
    v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(u32x4 q, float (&v)[4]) {  // fp32
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(q[i]);
}

// Rounded once to the dtype (nearest even).
template <bool NT = false>
__device__ __forceinline__ void store_piece(bf16_t* p, const float (&v)[8]) {
  u32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = uint32_t(f32_to_bf16(v[2 * i])) | (uint32_t(f32_to_bf16(v[2 * i + 1])) << 16);
  store_vec<NT, u32x4>(p, q);
}
template <bool NT = false>
__device__ __forceinline__ void store_piece(float* p, const float (&v)[4]) {
  store_vec<NT, f32x4>(p, f32x4{v[0], v[1], v[2], v[3]});
}

// Values of a piece kept in fp32.
__device__ __forceinline__ void store_f32(float* p, const float (&v)[4]) { store_piece(p, v); }
__device__ __forceinline__ void store_f32(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}

}  // namespace topmoe
