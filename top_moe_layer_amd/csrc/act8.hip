// Activations kept in 8 bits between the forward and the backward pass.
//
// Each group of 32 consecutive channels of a row (the row's last group may be
// shorter) shares one power-of-two scale 2^e and stores its elements as OCP
// e4m3 values q = x * 2^-e, rounded to nearest even: e is the smallest integer
// (at least -127) for which the group's largest finite magnitude is at most
// 448 * 2^e, 448 being e4m3's largest value, so nothing saturates and the
// scaling itself is exact.  The scale is stored as the byte e + 127.  An
// element that is not finite is stored as NaN and takes no part in the scale:
// a diverged activation stays visible in the gradients.
//
// One thread moves 16 bytes of an activation, 8 bf16 or 4 fp32 channels; the
// four or eight threads of a group find its largest magnitude with two or three
// lane exchanges.  SwiGLU with its two operands kept:
//   h  = SiLU(g) u          (from g, u as they came)
//   dg = dh u s (1 + g (1 - s)),  du = dh g s,  h = g s u,  s = sigmoid(g)
//                           (from the kept g, u; h for the down projection's
//                            weight gradient)
// Bound by memory: 16384 x 6464 bf16 on an MI355X, forward 137 us (854 MB, 6.2
// TB/s), backward 180 us (1.07 GB, 5.9 TB/s), no byte moved twice.  Inputs are
// read and kept bytes written non-temporally, the bytes being read again only
// in the backward pass: 147 us with neither, 144 with h alone written so.
#include "act8_impl.h"
#include "kernels.h"
#include "vec16.h"

#include "../../include/topmoe.h"

namespace topmoe {

namespace {

constexpr bool kNtLoad = true, kNtKeep = true;  // non-temporal, see above

__device__ __forceinline__ void load_q(const uint8_t* p, uint32_t (&q)[2]) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 v = load_vec<kNtLoad, u32x2>(p);
  q[0] = v.x;
  q[1] = v.y;
}
__device__ __forceinline__ void load_q(const uint8_t* p, uint32_t (&q)[1]) {
  q[0] = load_vec<kNtLoad, uint32_t>(p);
}
__device__ __forceinline__ void store_q(uint8_t* p, const uint32_t (&q)[2]) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  store_vec<kNtKeep, u32x2>(p, u32x2{q[0], q[1]});
}
__device__ __forceinline__ void store_q(uint8_t* p, const uint32_t (&q)[1]) {
  store_vec<kNtKeep, uint32_t>(p, q[0]);
}

// The thread's row and piece: pieces of E channels, a row's pieces padded to
// whole groups (pp = ceil(C / 32) groups of L lanes).
template <typename T>
struct Place {
  static constexpr int E = kE<T>, L = kGroupLanes<kE<T>>;
  int64_t r;
  int p;
  bool any, in;  // any: within the launch's rows; in: and within the row
  uint32_t groups;
  __device__ __forceinline__ Place(int64_t r0, uint32_t pieces, uint32_t pp, int C) {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    const uint32_t dr = i / pp;
    r = r0 + dr;
    p = int(i - dr * pp);
    any = i < pieces;
    in = any && p < C / E;
    groups = pp / L;
  }
  __device__ __forceinline__ int64_t at(int64_t pitch) const { return r * pitch + int64_t(p) * E; }
  __device__ __forceinline__ int64_t group() const { return r * groups + p / L; }
  __device__ __forceinline__ bool first() const { return any && p % L == 0; }
};

template <typename T>
__global__ __launch_bounds__(256) void act8_pack_kernel(const T* __restrict__ x, int64_t ldx,
                                                        int64_t r0, uint32_t pieces, uint32_t pp,
                                                        int C, uint8_t* __restrict__ q,
                                                        uint8_t* __restrict__ scale) {
  const Place<T> a(r0, pieces, pp, C);
  constexpr int E = kE<T>;
  float v[E];
  unpack(load_piece_if<kNtLoad>(a.in, x + a.at(ldx)), v);
  uint32_t b[E / 4];
  const uint32_t s = pack_q<E>(v, b);
  if (a.in) store_q(q + a.at(C), b);
  if (a.first()) scale[a.group()] = uint8_t(s);
}

template <typename T, bool NT>
__global__ __launch_bounds__(256) void act8_unpack_kernel(const uint8_t* __restrict__ q,
                                                          const uint8_t* __restrict__ scale,
                                                          int64_t r0, uint32_t pieces,
                                                          uint32_t pp, int C, T* __restrict__ x,
                                                          int64_t ldx) {
  const Place<T> a(r0, pieces, pp, C);
  constexpr int E = kE<T>;
  if (!a.in) return;
  uint32_t b[E / 4];
  load_q(q + a.at(C), b);
  float v[E];
  unpack_q<E>(b, scale_of(scale[a.group()]), v);
  store_piece<NT>(x + a.at(ldx), v);
}

template <typename T, bool NT>
__global__ __launch_bounds__(256) void swiglu_act8_fwd_kernel(
    const T* __restrict__ g, const T* __restrict__ u, int64_t ldg, int64_t ldu, int64_t r0,
    uint32_t pieces, uint32_t pp, int C, T* __restrict__ h, uint8_t* __restrict__ gq, uint8_t* __restrict__ gs,
    uint8_t* __restrict__ uq, uint8_t* __restrict__ us) {
  const Place<T> a(r0, pieces, pp, C);
  constexpr int E = kE<T>;
  float vg[E], vu[E], vh[E];
  unpack(load_piece_if<kNtLoad>(a.in, g + a.at(ldg)), vg);
  unpack(load_piece_if<kNtLoad>(a.in, u + a.at(ldu)), vu);
  uint32_t bg[E / 4], bu[E / 4];
  const uint32_t sg = pack_q<E>(vg, bg), su = pack_q<E>(vu, bu);
  const int64_t o = a.at(C);
  if (a.in) {
#pragma unroll
    for (int i = 0; i < E; ++i) vh[i] = silu(vg[i]) * vu[i];
    store_piece<NT>(h + o, vh);
    store_q(gq + o, bg);
    store_q(uq + o, bu);
  }
  if (a.first()) {
    gs[a.group()] = uint8_t(sg);
    us[a.group()] = uint8_t(su);
  }
}

template <typename T, bool NT>
__global__ __launch_bounds__(256) void swiglu_act8_bwd_kernel(
    const uint8_t* __restrict__ gq, const uint8_t* __restrict__ gs,
    const uint8_t* __restrict__ uq, const uint8_t* __restrict__ us, const T* __restrict__ dh,
    int64_t r0, uint32_t pieces, uint32_t pp, int C, T* __restrict__ dg,
    int64_t ldg, T* __restrict__ du, int64_t ldu, T* __restrict__ h) {
  const Place<T> a(r0, pieces, pp, C);
  constexpr int E = kE<T>;
  if (!a.in) return;
  const int64_t o = a.at(C), si = a.group();
  uint32_t bg[E / 4], bu[E / 4];
  load_q(gq + o, bg);
  load_q(uq + o, bu);
  float vg[E], vu[E], vd[E];
  const u32x4 raw = load_piece<kNtLoad>(dh + o);
  unpack_q<E>(bg, scale_of(gs[si]), vg);
  unpack_q<E>(bu, scale_of(us[si]), vu);
  unpack(raw, vd);
  float og[E], ou[E], oh[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float s = sigmoid(vg[i]), gsig = vg[i] * s;
    ou[i] = vd[i] * gsig;
    oh[i] = gsig * vu[i];
    og[i] = vd[i] * (vu[i] * s * (1.0f + vg[i] * (1.0f - s)));  // dh * u may pass the range
  }
  store_piece<NT>(dg + a.at(ldg), og);
  store_piece<NT>(du + a.at(ldu), ou);
  if (h != nullptr) store_piece<NT>(h + o, oh);
}

// ---- the (g, u) pairs of a training forward's workspace ----------------------
// A thread's pairs: 32 bytes, g in the low halves of bf16's words.
__device__ __forceinline__ void load_pairs(const bf16_t* p, float (&g)[8], float (&u)[8]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const u32x4 q = load_vec<true, u32x4>(p + 8 * w);
#pragma unroll
    for (int i = 0; i < 4; ++i) PairWord<bf16_t>::unpack(q[i], g[4 * w + i], u[4 * w + i]);
  }
}
__device__ __forceinline__ void load_pairs(const float* p, float (&g)[4], float (&u)[4]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const f32x4 q = load_vec<true, f32x4>(p + 4 * w);
    g[2 * w] = q.x; u[2 * w] = q.y;
    g[2 * w + 1] = q.z; u[2 * w + 1] = q.w;
  }
}

// pairs [R, C] (C a multiple of 64) to g and u in 8 bits (back: backward.hip).
template <typename T>
__global__ __launch_bounds__(256) void pairs_pack_kernel(
    const T* __restrict__ pairs, int64_t r0, uint32_t pieces, uint32_t pp, int C,
    uint8_t* __restrict__ gq, uint8_t* __restrict__ gs, uint8_t* __restrict__ uq,
    uint8_t* __restrict__ us) {
  const Place<T> a(r0, pieces, pp, C);
  constexpr int E = kE<T>;
  const int64_t o = a.at(C);
  float g[E], u[E];
  if (a.in) {
    load_pairs(pairs + 2 * o, g, u);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) g[i] = u[i] = 0.f;
  }
  uint32_t bg[E / 4], bu[E / 4];
  const uint32_t sg = pack_q<E>(g, bg), su = pack_q<E>(u, bu);
  if (!a.in) return;
  store_q(gq + o, bg);
  store_q(uq + o, bu);
  if (a.first()) {
    gs[a.group()] = uint8_t(sg);
    us[a.group()] = uint8_t(su);
  }
}

// 16 bytes a thread.
__global__ __launch_bounds__(256) void copy_kernel(const u32x4* __restrict__ src,
                                                   u32x4* __restrict__ dst, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256)
    dst[i] = src[i];
}

// Launches over slabs of rows of at most 2^30 pieces, so that piece numbers
// stay in 32 bits and a grid within its limit of threads.
template <typename T, typename F>
hipError_t for_slabs(int64_t R, int64_t C, const Launch& s, F launch) {
  const uint32_t pp = uint32_t((C + kAct8Group - 1) / kAct8Group * Place<T>::L);
  int64_t slab = (int64_t(1) << 30) / pp;
  if (slab < 1) slab = 1;
  for (int64_t r0 = 0; r0 < R; r0 += slab) {
    Launch L = s;
    if (r0 > 0) L.start = nullptr;
    if (r0 + slab < R) L.stop = nullptr;
    const int64_t rows = r0 + slab < R ? slab : R - r0;
    const uint32_t pieces = uint32_t(rows * pp);
    const hipError_t e = launch(dim3((pieces + 255) / 256), r0, pieces, pp, L);
    if (e != hipSuccess) return e;
    s.launched = true;
  }
  return hipSuccess;
}

}  // namespace

#define TOPMOE_ACT8(T, KERNEL, ...)                                                                \
  for_slabs<T>(R, C, s, [&](dim3 grid, int64_t r0, uint32_t pieces, uint32_t pp, const Launch& L) { \
    return launch_kernel(KERNEL, grid, dim3(256), 0, L, __VA_ARGS__);                              \
  })
// KERNEL<T, NT> by the outputs' bytes.
#define TOPMOE_ACT8_NT(T, KERNEL, BYTES, ...)                                 \
  return (BYTES) >= kNtBytes ? TOPMOE_ACT8(T, (KERNEL<T, true>), __VA_ARGS__) \
                             : TOPMOE_ACT8(T, (KERNEL<T, false>), __VA_ARGS__)

namespace {

template <typename T>
hipError_t unpack_typed(const uint8_t* q, const uint8_t* scale, int64_t R, int64_t C, void* x,
                  int64_t ldx, const Launch& s) {
  TOPMOE_ACT8_NT(T, act8_unpack_kernel, R * C * int64_t(sizeof(T)), q, scale, r0, pieces, pp,
                 int(C), static_cast<T*>(x), ldx);
}

template <typename T>
hipError_t swiglu_fwd(const void* g, int64_t ldg, const void* u, int64_t ldu, int64_t R,
                      int64_t C, void* h, uint8_t* gq, uint8_t* gs, uint8_t* uq, uint8_t* us,
                      const Launch& s) {
  TOPMOE_ACT8_NT(T, swiglu_act8_fwd_kernel, R * C * int64_t(sizeof(T)),
                 static_cast<const T*>(g), static_cast<const T*>(u), ldg, ldu, r0, pieces, pp,
                 int(C), static_cast<T*>(h), gq, gs, uq, us);
}

template <typename T>
hipError_t swiglu_bwd(const uint8_t* gq, const uint8_t* gs, const uint8_t* uq, const uint8_t* us,
                      const void* dh, int64_t R, int64_t C, void* dg, int64_t ldg, void* du,
                      int64_t ldu, void* h, const Launch& s) {
  TOPMOE_ACT8_NT(T, swiglu_act8_bwd_kernel, R * C * int64_t(sizeof(T)) * (h != nullptr ? 3 : 2),
                 gq, gs, uq, us, static_cast<const T*>(dh), r0, pieces, pp, int(C),
                 static_cast<T*>(dg), ldg, static_cast<T*>(du), ldu, static_cast<T*>(h));
}

}  // namespace

hipError_t launch_act8_pack(const void* x, int64_t ldx, int64_t R, int64_t C, int dtype,
                            uint8_t* q, uint8_t* scale, const Launch& s) {
  if (dtype == TOPMOE_DTYPE_FP32)
    return TOPMOE_ACT8(float, act8_pack_kernel<float>, static_cast<const float*>(x), ldx, r0, pieces, pp,
                       int(C), q, scale);
  return TOPMOE_ACT8(bf16_t, act8_pack_kernel<bf16_t>, static_cast<const bf16_t*>(x), ldx, r0, pieces, pp,
                     int(C), q, scale);
}

hipError_t launch_act8_unpack(const uint8_t* q, const uint8_t* scale, int64_t R, int64_t C,
                              int dtype, void* x, int64_t ldx, const Launch& s) {
  return dtype == TOPMOE_DTYPE_FP32 ? unpack_typed<float>(q, scale, R, C, x, ldx, s)
                                    : unpack_typed<bf16_t>(q, scale, R, C, x, ldx, s);
}

hipError_t launch_swiglu_act8_fwd(const void* g, int64_t ldg, const void* u, int64_t ldu,
                                  int64_t R, int64_t C, int dtype, void* h, uint8_t* gq,
                                  uint8_t* gs, uint8_t* uq, uint8_t* us, const Launch& s) {
  return dtype == TOPMOE_DTYPE_FP32
             ? swiglu_fwd<float>(g, ldg, u, ldu, R, C, h, gq, gs, uq, us, s)
             : swiglu_fwd<bf16_t>(g, ldg, u, ldu, R, C, h, gq, gs, uq, us, s);
}

hipError_t launch_swiglu_act8_bwd(const uint8_t* gq, const uint8_t* gs, const uint8_t* uq,
                                  const uint8_t* us, const void* dh, int64_t R, int64_t C,
                                  int dtype, void* dg, int64_t ldg, void* du, int64_t ldu, void* h,
                                  const Launch& s) {
  return dtype == TOPMOE_DTYPE_FP32
             ? swiglu_bwd<float>(gq, gs, uq, us, dh, R, C, dg, ldg, du, ldu, h, s)
             : swiglu_bwd<bf16_t>(gq, gs, uq, us, dh, R, C, dg, ldg, du, ldu, h, s);
}

hipError_t launch_pairs_pack(const void* pairs, int64_t R, int64_t C, int dtype, uint8_t* gq,
                             uint8_t* gs, uint8_t* uq, uint8_t* us, const Launch& s) {
  if (dtype == TOPMOE_DTYPE_FP32)
    return TOPMOE_ACT8(float, pairs_pack_kernel<float>, static_cast<const float*>(pairs), r0, pieces, pp,
                       int(C), gq, gs, uq, us);
  return TOPMOE_ACT8(bf16_t, pairs_pack_kernel<bf16_t>, static_cast<const bf16_t*>(pairs), r0, pieces, pp,
                     int(C), gq, gs, uq, us);
}

hipError_t launch_copy(const void* src, void* dst, size_t bytes, const Launch& s) {
  const int64_t n = int64_t(bytes / 16);
  if (n == 0) return hipSuccess;
  const int64_t grid = (n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096;
  return launch_kernel(copy_kernel, dim3(unsigned(grid)), dim3(256), 0, s,
                       static_cast<const u32x4*>(src), static_cast<u32x4*>(dst), n);
}

#undef TOPMOE_ACT8
#undef TOPMOE_ACT8_NT

}  // namespace topmoe
