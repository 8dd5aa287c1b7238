// The RMS norms before and after a block, fused with the block's gate, its
// residual stream and the residual's scale; forward and backward.
//
// Per token (row of H channels), all in fp32:
//   after   yh = y * rstd_y,  rstd_y = 1 / sqrt(mean(y^2) + eps)   (no norm: yh = y, w = 1)
//           r  = s * residual + gate * w * yh,   out = round(r)
//   before  n  = round(r * rstd_r * w_next),  rstd_r = 1 / sqrt(mean(r^2) + eps)
// A pre-norm alone is the second line with r = x.  Gradients, with
// rh = out * rstd_r and a = dn * w_next:
//   dr   = dout + rstd_r * (a - rh * mean(a * rh)),      dw_next = sum_t dn * rh
//   dres = s * dr,   b = dr * gate * w
//   dy   = rstd_y * (b - yh * mean(b * yh))  (no norm: b)
//   dw   = sum_t gate * dr * yh,   dgate = the sum of w * dr * yh over what shares the gate
//
// R threads per row, V pieces of 16 bytes each: a block of R / 64 wavefronts,
// or for narrow rows a wavefront or a part of one, 256 / R rows a block.  The
// row stays in registers between its statistics and its use, so every tensor
// is read once and written once.  Bound by memory: post norm with a channel
// gate and the next norm, 16384 x 2048 bf16 on an MI355X, 46 us forward (268
// MB, 5.8 TB/s) and 78 us backward (402 MB; rows 71 us with their partial sums
// at 5.9 TB/s, then the sums).
//
// Column sums of the backward pass (dw, dgate, dw_next) are taken in two fixed
// steps without atomics: each unit of consecutive rows sums its own rows in
// registers and writes one fp32 row of partial sums; a second launch adds the
// units' rows in order.  A channel gate may have G rows, each shared by
// N / G consecutive tokens: units either lie within one such group (their
// partial sums are of dr * yh, weighted by the gate and by w afterwards), or
// hold whole groups, whose dgate they then write themselves (the partial sums
// are of gate * dr * yh).
#include "kernels.h"
#include "vec16.h"

#include "../../include/topmoe.h"

namespace topmoe {

namespace {

// Rows a block holds side by side, and wavefronts of a row.
template <int R>
constexpr int kSide = R <= 64 ? 256 / R : 1;
template <int R>
constexpr int kWaves = R <= 64 ? 1 : R / 64;
template <int R>
constexpr int kThreads = R <= 64 ? 256 : R;

// Sum over a row's R threads, lanes as a butterfly and wavefronts in order.
// `slot` (2 x W floats of LDS) alternates between calls: a wavefront writing a
// slot again has passed the barrier of the call in between, which every reader
// of the slot's last use reached after reading it.
template <int R, int W = kWaves<R>>
__device__ __forceinline__ float row_sum(float v, float (&slot)[2][W], int& turn, int wave) {
#pragma unroll
  for (int o = R < 64 ? R / 2 : 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) slot[turn][wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += slot[turn][i];
    turn ^= 1;
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void load_f(const T* p, float (&v)[kE<T>]) {
  unpack(load_piece(p), v);
}

// POST: the norm after the block with gate and residual (else r = y = x).
// NEXT: the norm before the next block.  NT: non-temporal rows (see kNtBytes;
// the rows read as well: 48.3 -> 45.7 us of the 16384 x 2048 post norm).
template <typename T, int R, int V, bool POST, bool NEXT, bool NT>
__global__ __launch_bounds__(kThreads<R>) void norm_fwd_kernel(NormFwd a) {
  constexpr int E = kE<T>;
  __shared__ float slot[2][kWaves<R>];
  const int lane = int(threadIdx.x) % R, wave = int(threadIdx.x >> 6);
  const int64_t t = a.t0 + int64_t(blockIdx.x) * kSide<R> + int(threadIdx.x) / R;
  if (kSide<R> > 1 && t >= a.N) return;
  int turn = 0;
  const T* y = static_cast<const T*>(a.y) + t * a.H;
  u32x4 yr[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = lane + v * R;
    yr[v] = load_piece_if<NT>(p < a.hv, y + p * E);
  }
  const float inv_h = 1.0f / float(a.H);
  float rs[V][E];  // r
  if constexpr (POST) {
    u32x4 res[V];
    const T* rp = static_cast<const T*>(a.residual) + t * a.H;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = lane + v * R;
      res[v] = load_piece_if<NT>(p < a.hv, rp + p * E);
    }
    float rstd = 1.f;
    if (a.w != nullptr) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[E];
        unpack(yr[v], f);
#pragma unroll
        for (int c = 0; c < E; ++c) s = fmaf(f[c], f[c], s);
      }
      rstd = 1.0f / sqrtf(row_sum<R>(s, slot, turn, wave) * inv_h + a.eps);
      if (lane == 0) a.rstd[t] = rstd;
    }
    float gt = 1.f;
    const T* gp = nullptr;
    if (a.gate_mode == kGateToken) gt = to_f32<T>(static_cast<const T*>(a.gate)[t]);
    if (a.gate_mode == kGateChannel) gp = static_cast<const T*>(a.gate) + (t / a.gate_span) * a.H;
    T* out = static_cast<T*>(a.out) + t * a.H;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = lane + v * R;
      float f[E], q[E];
      unpack(yr[v], f);
      unpack(res[v], q);
      if (p < a.hv) {
        float m[E];
#pragma unroll
        for (int c = 0; c < E; ++c) m[c] = rstd * gt;
        if (a.w != nullptr) {
          float w[E];
          load_f<T>(static_cast<const T*>(a.w) + p * E, w);
#pragma unroll
          for (int c = 0; c < E; ++c) m[c] *= w[c];
        }
        if (gp != nullptr) {
          float g[E];
          load_f<T>(gp + p * E, g);
#pragma unroll
          for (int c = 0; c < E; ++c) m[c] *= g[c];
        }
#pragma unroll
        for (int c = 0; c < E; ++c) rs[v][c] = fmaf(f[c], m[c], a.scale * q[c]);
        store_piece<NT>(out + p * E, rs[v]);
      } else {
#pragma unroll
        for (int c = 0; c < E; ++c) rs[v][c] = 0.f;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) unpack(yr[v], rs[v]);
  }
  if constexpr (NEXT) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int c = 0; c < E; ++c) s = fmaf(rs[v][c], rs[v][c], s);
    const float rstd = 1.0f / sqrtf(row_sum<R>(s, slot, turn, wave) * inv_h + a.eps);
    if (lane == 0) a.next_rstd[t] = rstd;
    T* n = static_cast<T*>(a.n) + t * a.H;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = lane + v * R;
      if (p >= a.hv) continue;
      float w[E];
      load_f<T>(static_cast<const T*>(a.next_w) + p * E, w);
#pragma unroll
      for (int c = 0; c < E; ++c) w[c] = rs[v][c] * rstd * w[c];
      store_piece<NT>(n + p * E, w);
    }
  }
}

// What one row of the backward pass reads, as loaded.
template <int V>
struct BwdRow {
  u32x4 dout[V], y[V], out[V], dn[V];
  float rstd, next_rstd, gate;  // gate: of a token gate
};

template <typename T, int R, int V, bool POST, bool NEXT>
__device__ __forceinline__ void load_row(const NormBwd& a, int64_t t, int lane,
                                         BwdRow<V>& r) {
  constexpr int E = kE<T>;
  const int64_t row = t * a.H;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = lane + v * R;
    const bool in = p < a.hv;
    const int64_t at = row + p * E;
    if constexpr (NEXT) {
      r.out[v] = load_piece_if<true>(in, static_cast<const T*>(a.out) + at);
      r.dn[v] = load_piece_if<true>(in, static_cast<const T*>(a.dn) + at);
    }
    r.dout[v] = load_piece_if<true>(in && a.dout != nullptr, static_cast<const T*>(a.dout) + at);
    if constexpr (POST)
      r.y[v] = load_piece_if<true>(in, static_cast<const T*>(a.y) + at);
  }
  if constexpr (NEXT) r.next_rstd = a.next_rstd[t];
  if constexpr (POST) {
    r.rstd = a.rstd != nullptr ? a.rstd[t] : 1.f;
    r.gate = a.gate_mode == kGateToken ? to_f32<T>(static_cast<const T*>(a.gate)[t]) : 1.f;
  }
}

// One unit of rows per block (see NormUnits): row gradients, and the unit's
// column sums in registers.  FLUSH: units of whole gate groups.  PRE: the
// weights stay in registers, and the next row's loads are issued before a
// row's sums, so that they run under its barriers; the widest rows have no
// registers left for that and load what they need when they need it.  With both
// norms fp32 rows above 8192 channels spill even so, 57 registers (87 with whole
// groups; bf16 2 and 43): 1365 x 12288 fp32 reads 428 MB and writes 245 for 268
// and 159, in 141 us; 2730 x 12288 bf16 takes 92.  One norm takes 45 to 55 us
// above 8192 channels (201 or 268 MB).  The
// residual's gradient, which nobody reads before the block's own backward pass
// is through, is written non-temporally (NT) once it and dy fill half the
// Infinity Cache (16384 x 2048 bf16: 80.0 -> 77.3 us, with readers of both
// behind 124.3 -> 119.4, at half the rows 67.5 -> 69.1; dy as well: 86.9).  The units
// side by side in a block of narrow rows add their sums to one partial row.
template <typename T, int R, int V, bool POST, bool NEXT, bool FLUSH, bool PRE, bool NT>
__global__ __launch_bounds__(kThreads<R>) void norm_bwd_kernel(NormBwd a) {
  constexpr int E = kE<T>, G = kSide<R>;
  __shared__ float slot[2][kWaves<R>];
  const int wave = int(threadIdx.x >> 6), side = int(threadIdx.x) / R;
  const int lane = int(threadIdx.x) % R;
  int turn = 0;
  const float inv_h = 1.0f / float(a.H);
  const int64_t unit = int64_t(blockIdx.x) * G + side;
  int64_t r0, r1, group = 0;
  if constexpr (!FLUSH) {  // a piece of one gate group
    group = unit / a.units.per_group;
    r0 = group * a.gate_span + (unit - group * a.units.per_group) * a.units.rows;
    const int64_t end = (group + 1) * a.gate_span;
    r1 = r0 + a.units.rows < end ? r0 + a.units.rows : end;
  } else {
    r0 = unit * a.units.rows;
    r1 = r0 + a.units.rows < a.N ? r0 + a.units.rows : a.N;
    group = r0 / a.gate_span;
  }
  const bool any = r0 < r1;  // a block's last units may have no rows
  const T* cgate = POST && any && a.gate_mode == kGateChannel
                       ? static_cast<const T*>(a.gate) + group * a.H : nullptr;
  u32x4 w[V], nw[V], cg[V];  // PRE: post and next weight, the current group's gate
  auto hold = [&](u32x4(&r)[V], const void* from) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = lane + v * R;
      r[v] = load_piece_if(from != nullptr && p < a.hv, static_cast<const T*>(from) + p * E);
    }
  };
  auto held = [&](const u32x4& r, const void* from, int p, float(&f)[E]) {
    if constexpr (PRE) unpack(r, f);
    else unpack(load_piece_if(p < a.hv, static_cast<const T*>(from) + p * E), f);
  };
  if constexpr (PRE) {
    if constexpr (NEXT) hold(nw, a.next_w);
    if constexpr (POST) {
      hold(w, a.w);
      hold(cg, cgate);
    }
  }
  float sg[V][E], sn[V][E];   // sums for dgate and dw (of the current group), dw_next
  float sw[FLUSH ? V : 1][E];  // for dw, of the finished groups
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int c = 0; c < E; ++c) {
      sg[v][c] = sn[v][c] = 0.f;
      if constexpr (FLUSH) sw[v][c] = 0.f;
    }

  BwdRow<V> cur;
  if (PRE && any) load_row<T, R, V, POST, NEXT>(a, r0, lane, cur);
  int64_t left = FLUSH ? a.gate_span : 0;  // rows to the end of the group
  for (int64_t t = r0; t < r1; ++t) {
    BwdRow<V> nxt;
    if constexpr (PRE) load_row<T, R, V, POST, NEXT>(a, t + 1 < r1 ? t + 1 : t, lane, nxt);
    else load_row<T, R, V, POST, NEXT>(a, t, lane, cur);
    float dr[V][E];
#pragma unroll
    for (int v = 0; v < V; ++v) unpack(cur.dout[v], dr[v]);
    if constexpr (NEXT) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float rh[E], av[E], wv[E];
        unpack(cur.out[v], rh);
        unpack(cur.dn[v], av);
        held(nw[v], a.next_w, lane + v * R, wv);
#pragma unroll
        for (int c = 0; c < E; ++c) {
          rh[c] *= cur.next_rstd;
          sn[v][c] = fmaf(av[c], rh[c], sn[v][c]);
          s = fmaf(av[c] * wv[c], rh[c], s);
        }
      }
      const float m = row_sum<R>(s, slot, turn, wave) * inv_h;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float rh[E], av[E], wv[E];
        unpack(cur.out[v], rh);
        unpack(cur.dn[v], av);
        held(nw[v], a.next_w, lane + v * R, wv);
#pragma unroll
        for (int c = 0; c < E; ++c)
          dr[v][c] += cur.next_rstd * (av[c] * wv[c] - rh[c] * cur.next_rstd * m);
      }
    }
    if constexpr (!POST) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int p = lane + v * R;
        if (p < a.hv) store_piece(static_cast<T*>(a.dy) + t * a.H + p * E, dr[v]);
      }
    } else {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int p = lane + v * R;
        float q[E], yh[E], g[E];
        unpack(cur.y[v], yh);
#pragma unroll
        for (int c = 0; c < E; ++c) {
          q[c] = a.scale * dr[v][c];
          yh[c] *= cur.rstd;
          sg[v][c] = fmaf(dr[v][c] * cur.gate, yh[c], sg[v][c]);
        }
        if (p < a.hv) store_piece<NT>(static_cast<T*>(a.dresidual) + t * a.H + p * E, q);
        if (a.w != nullptr) {  // from here dr is b without a token gate
          held(w[v], a.w, p, g);
#pragma unroll
          for (int c = 0; c < E; ++c) dr[v][c] *= g[c];
        }
        if (cgate != nullptr) {
          held(cg[v], cgate, p, g);
#pragma unroll
          for (int c = 0; c < E; ++c) dr[v][c] *= g[c];
        }
#pragma unroll
        for (int c = 0; c < E; ++c) s = fmaf(dr[v][c], yh[c], s);
      }
      float m = 0.f;
      if (a.w != nullptr || a.gate_mode == kGateToken) {
        s = row_sum<R>(s, slot, turn, wave);
        if (a.gate_mode == kGateToken && lane == 0)
          static_cast<T*>(a.dgate)[t] = from_f32<T>(s);
        m = a.w != nullptr ? s * inv_h : 0.f;
      }
      const float k = cur.gate * cur.rstd;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int p = lane + v * R;
        float yh[E];
        unpack(cur.y[v], yh);
#pragma unroll
        for (int c = 0; c < E; ++c) yh[c] = k * (dr[v][c] - yh[c] * cur.rstd * m);
        if (p < a.hv) store_piece(static_cast<T*>(a.dy) + t * a.H + p * E, yh);
      }
      if constexpr (FLUSH) {
        if (--left == 0) {  // the group ends
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const int p = lane + v * R;
            float g[E], q[E];
            held(cg[v], cgate, p, g);
            if (a.w != nullptr) held(w[v], a.w, p, q);
#pragma unroll
            for (int c = 0; c < E; ++c) {
              sw[v][c] = fmaf(g[c], sg[v][c], sw[v][c]);
              q[c] = a.w != nullptr ? q[c] * sg[v][c] : sg[v][c];
              sg[v][c] = 0.f;
            }
            if (p < a.hv) store_piece(static_cast<T*>(a.dgate) + group * a.H + p * E, q);
          }
          left = a.gate_span;
          ++group;
          cgate += a.H;
          if (PRE && t + 1 < r1) hold(cg, cgate);
        }
      }
    }
    if constexpr (PRE) cur = nxt;
  }
  // One partial row per block: the units' sums added in order.
  __shared__ float sums[G > 1 ? G - 1 : 1][G > 1 ? R * V * E : 1];
  auto out = [&](float(&acc)[V][E], float* part) {
    if constexpr (G > 1) {
      __syncthreads();
      if (side > 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int c = 0; c < E; ++c) sums[side - 1][(v * E + c) * R + lane] = acc[v][c];
      }
      __syncthreads();
      if (side > 0) return;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int c = 0; c < E; ++c)
          for (int g = 0; g < G - 1; ++g) acc[v][c] += sums[g][(v * E + c) * R + lane];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = lane + v * R;
      if (p < a.hv) store_f32(part + int64_t(blockIdx.x) * a.H + p * E, acc[v]);
    }
  };
  if constexpr (POST) {
    if (a.part != nullptr) {
      if constexpr (FLUSH) out(sw, a.part);
      else out(sg, a.part);
    }
  }
  if constexpr (NEXT) out(sn, a.part_next);
}

// Column sums of the blocks' partial rows.  Role 0: dw, and dgate of a gate with
// one row, from the same sums; 1: dw_next; 2 + g: row g of a gate with several.
// 32 channels a block; slice s of 32 adds rows s, s + 32, ..., eight loads in
// flight, and the 32 sums are added in order.
template <typename T>
__global__ __launch_bounds__(1024) void norm_reduce_kernel(NormBwd a) {
  __shared__ float sm[32][32];
  const int col = threadIdx.x & 31, s = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + col;
  const bool in = h < a.H;
  const int role = a.first_role + int(blockIdx.y);
  const float* part = (role == 1 ? a.part_next : a.part) + (in ? h : 0);
  const int64_t per_group = a.units.per_group / a.units.blocks_of;
  int64_t u0 = 0, u1 = a.units.count / a.units.blocks_of;
  if (role >= 2) {
    u0 = int64_t(role - 2) * per_group;
    u1 = u0 + per_group < u1 ? u0 + per_group : u1;  // no units: sums of nothing
  }
  // several gate rows: dw adds each unit's sums times its group's gate
  const bool gated = role == 0 && a.gate_mode == kGateChannel && a.units.per_group > 0 &&
                     a.gate_rows > 1;
  const T* gate = static_cast<const T*>(a.gate) + (in ? h : 0);
  // x / per_group as x * ceil(2^28 / per_group) >> 28, exact for both below 2^14:
  // plans of several gate rows that get here have fewer than 2^13 blocks.
  const uint64_t magic = gated ? ((1u << 28) + uint32_t(per_group) - 1) / uint32_t(per_group) : 0;
  float acc = 0.f;
  for (int64_t u = u0 + s; u < u1; u += 32 * 8) {
    float v[8];
    T g[8];  // converted only after all loads are on their way
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t x = u + i * 32;
      v[i] = x < u1 ? part[x * a.H] : 0.f;
    }
    if (gated) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t x = u + i * 32 < u1 ? u + i * 32 : u1 - 1;
        g[i] = gate[int64_t(uint32_t(x) * magic >> 28) * a.H];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = u + i * 32 < u1 ? v[i] * to_f32<T>(g[i]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc += v[i];
  }
  sm[s][col] = acc;
  __syncthreads();
  if (s != 0 || !in) return;
  acc = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) acc += sm[i][col];
  if (role == 1) {
    static_cast<T*>(a.dnext_w)[h] = from_f32<T>(acc);
    return;
  }
  const bool one = role == 0 && a.gate_mode == kGateChannel && a.units.per_group > 0 &&
                   a.gate_rows == 1;  // an empty batch's gate may have no row at all
  if (role >= 2 || one) {
    const float w = a.w != nullptr ? to_f32<T>(static_cast<const T*>(a.w)[h]) : 1.f;
    static_cast<T*>(a.dgate)[int64_t(role >= 2 ? role - 2 : 0) * a.H + h] = from_f32<T>(acc * w);
  }
  if (role == 0 && a.dw != nullptr)
    static_cast<T*>(a.dw)[h] = from_f32<T>(one ? acc * to_f32<T>(gate[0]) : acc);
}

// dgate of many rows from few units each: a thread per value, its units' sums
// added in order, eight loads in flight.  In a launch of its own from 2^16 values
// on: 128 rows, 4096 x 16384 bf16, 286 -> 114 us; 32 rows, 16384 x 2048, 68 ->
// 61; for 8 rows of 2048 the launch would cost more than it saves (21 / 22).
constexpr int kFewUnits = 32;
constexpr int64_t kManyValues = int64_t(1) << 16;

template <typename T>
__global__ __launch_bounds__(256) void norm_gate_sums_kernel(NormBwd a) {
  const int h = int(blockIdx.x) * 256 + int(threadIdx.x);
  if (h >= a.H) return;
  const int64_t g = blockIdx.y;
  const int units = int(a.units.per_group / a.units.blocks_of);
  const float* part = a.part + g * units * a.H + h;
  float acc = 0.f;
  for (int u = 0; u < units; u += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u + i < units ? part[int64_t(u + i) * a.H] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc += v[i];
  }
  const float w = a.w != nullptr ? to_f32<T>(static_cast<const T*>(a.w)[h]) : 1.f;
  static_cast<T*>(a.dgate)[g * a.H + h] = from_f32<T>(acc * w);
}

template <typename T, int R, int V>
hipError_t fwd_flags(const NormFwd& a, bool post, bool next, int64_t rows, const Launch& L) {
  const dim3 grid(unsigned((rows + kSide<R> - 1) / kSide<R>)), block(kThreads<R>);
  const bool nt = a.N * a.H * int64_t(sizeof(T)) * (post && next ? 2 : 1) >= kNtBytes;
#define TOPMOE_NORM_FWD(POST, NEXT)                                                               \
  return nt ? launch_kernel(norm_fwd_kernel<T, R, V, POST, NEXT, true>, grid, block, 0, L, a) \
            : launch_kernel(norm_fwd_kernel<T, R, V, POST, NEXT, false>, grid, block, 0, L, a)
  if (post && next) TOPMOE_NORM_FWD(true, true);
  if (post) TOPMOE_NORM_FWD(true, false);
  TOPMOE_NORM_FWD(false, true);
#undef TOPMOE_NORM_FWD
}

template <typename T>
hipError_t fwd_typed(NormFwd a, bool post, bool next, const Launch& s) {
  // rows of one launch: at most 2^21, so that a grid of 1024 threads a row keeps
  // below 2^32 threads
  const int64_t slab = int64_t(1) << 21, N = a.N;
  for (int64_t t0 = 0; t0 < N; t0 += slab) {
    Launch L = s;
    if (t0 > 0) L.start = nullptr;
    if (t0 + slab < N) L.stop = nullptr;
    a.t0 = t0;
    const int64_t rows = t0 + slab < N ? slab : N - t0;
    hipError_t e = hipErrorInvalidValue;
    // Pieces in use by all lanes, two or more loads in flight each, and few
    // barriers: against 4 wavefronts for every H above 512 and one below,
    // the bytes of 16384 x 2048 take 50 / 46 (H = 2048: 256 x 1 against 128 x 2),
    // 83 / 50 (768), 83 / 48 (256) and 273 / 50 us (64).
    if (a.hv <= 8) e = fwd_flags<T, 8, 1>(a, post, next, rows, L);
    else if (a.hv <= 16) e = fwd_flags<T, 16, 1>(a, post, next, rows, L);
    else if (a.hv <= 32) e = fwd_flags<T, 32, 1>(a, post, next, rows, L);
    else if (a.hv <= 64) e = fwd_flags<T, 64, 1>(a, post, next, rows, L);
    else if (a.hv <= 128) e = fwd_flags<T, 64, 2>(a, post, next, rows, L);
    else if (a.hv <= 256) e = fwd_flags<T, 128, 2>(a, post, next, rows, L);
    else if (a.hv <= 512) e = fwd_flags<T, 256, 2>(a, post, next, rows, L);
    else if (a.hv <= 1024) e = fwd_flags<T, 256, 4>(a, post, next, rows, L);
    else if (kE<T> == 8 || a.hv <= 2048) e = fwd_flags<T, 512, 4>(a, post, next, rows, L);
    else if constexpr (kE<T> == 4) e = fwd_flags<T, 1024, 4>(a, post, next, rows, L);
    if (e != hipSuccess) return e;
    s.launched = true;
  }
  return hipSuccess;
}

template <typename T, int R, int V, bool POST, bool NEXT, bool PRE>
hipError_t bwd_kernel(const NormBwd& a, const Launch& L) {
  const dim3 grid(static_cast<unsigned>(a.units.count / a.units.blocks_of)), block(kThreads<R>);
#define TOPMOE_NORM_BWD(FLUSH, NT) \
  return launch_kernel(norm_bwd_kernel<T, R, V, POST, NEXT, FLUSH, PRE, NT>, grid, block, 0, L, a)
  if constexpr (POST) {
    const bool nt = 2 * a.N * a.H * int64_t(sizeof(T)) >= kNtBytes;
    if (a.units.per_group == 0) {
      if (nt) TOPMOE_NORM_BWD(true, true);
      TOPMOE_NORM_BWD(true, false);
    }
    if (nt) TOPMOE_NORM_BWD(false, true);
  }
  TOPMOE_NORM_BWD(false, false);
#undef TOPMOE_NORM_BWD
}

template <typename T, int R, int V, bool PRE>
hipError_t bwd_flags(const NormBwd& a, bool post, bool next, const Launch& L) {
  if (!post) return bwd_kernel<T, R, V, false, true, PRE>(a, L);
  if (next) return bwd_kernel<T, R, V, true, true, PRE>(a, L);
  return bwd_kernel<T, R, V, true, false, PRE>(a, L);
}

// Rows of 513 to 1024 pieces.  Both norms of eight channels a piece leave 1024
// threads no registers for the next row (H = 8192: 93 us loading each row when
// it is needed, 84 with spilled registers, 79 with 512 threads), 768 threads
// have them (H = 4200: 93 -> 84 us, 5944: 84 -> 81; with one norm, or between
// the other widths' threads, as many idle lanes less gave nothing).
template <typename T>
hipError_t bwd_upto_1024(const NormBwd& a, bool post, bool next, const Launch& L) {
  if constexpr (kE<T> == 4) {
    return bwd_flags<T, 1024, 1, true>(a, post, next, L);
  } else {
    if (post && next && a.hv <= 768) return bwd_kernel<T, 768, 1, true, true, true>(a, L);
    if (post && next) return bwd_kernel<T, 512, 2, true, true, true>(a, L);
    if (post) return bwd_kernel<T, 1024, 1, true, false, true>(a, L);
    return bwd_kernel<T, 1024, 1, false, true, true>(a, L);
  }
}

template <typename T>
hipError_t bwd_typed(const NormBwd& a, bool post, bool next, const Launch& rows,
                     const Launch& sums) {
  if (a.units.count > 0) {
    hipError_t e = hipErrorInvalidValue;
    // One piece a thread leaves registers for the next row's (H = 2048: 94 ->
    // 82 us); 128 threads for H = 1024 against 64 with two pieces: 81 / 88 us.
    if (a.hv <= 8) e = bwd_flags<T, 8, 1, true>(a, post, next, rows);
    else if (a.hv <= 16) e = bwd_flags<T, 16, 1, true>(a, post, next, rows);
    else if (a.hv <= 32) e = bwd_flags<T, 32, 1, true>(a, post, next, rows);
    else if (a.hv <= 64) e = bwd_flags<T, 64, 1, true>(a, post, next, rows);
    else if (a.hv <= 128) e = bwd_flags<T, 128, 1, true>(a, post, next, rows);
    else if (a.hv <= 256) e = bwd_flags<T, 256, 1, true>(a, post, next, rows);
    else if (a.hv <= 512) e = bwd_flags<T, 512, 1, true>(a, post, next, rows);
    else if (a.hv <= 1024) e = bwd_upto_1024<T>(a, post, next, rows);
    else if (kE<T> == 8 || a.hv <= 2048) e = bwd_flags<T, 1024, 2, false>(a, post, next, rows);
    else if constexpr (kE<T> == 4) e = bwd_flags<T, 1024, 4, false>(a, post, next, rows);
    if (e != hipSuccess) return e;
  }
  // The roles of the sums; neighbouring ones share a launch.  With tokens there
  // are fewer than 4096 gate rows (see plan_norm_units: more are written by units
  // of whole groups); an empty batch's may be more than a grid has rows.
  const bool channel = post && a.gate_mode == kGateChannel && a.units.per_group > 0;
  const bool first_role = post && (a.dw != nullptr || (channel && a.gate_rows == 1));
  const int64_t gates = channel && a.gate_rows > 1 ? a.gate_rows : 0;
  const int64_t first = first_role ? 0 : next ? 1 : 2;
  const int64_t end = gates > 0 ? 2 + gates : next ? 2 : first_role ? 1 : 0;
  const bool few = a.units.count > 0 && gates * a.H >= kManyValues &&
                   a.units.per_group <= kFewUnits * a.units.blocks_of;
  Launch L = sums;
  for (int64_t r = first; r < end;) {
    if (r == 1 && !next) {
      r = 2;
      continue;
    }
    int64_t stop = r == 0 && !next ? 1 : r < 2 && few && end > 2 ? 2 : end;
    if (stop - r > 65535) stop = r + 65535;
    L.stop = stop == end ? sums.stop : nullptr;
    NormBwd b = a;
    b.first_role = int(r);
    const unsigned roles = unsigned(stop - r);
    const hipError_t e =
        r >= 2 && few
            ? launch_kernel(norm_gate_sums_kernel<T>, dim3(unsigned((a.H + 255) / 256), roles),
                            dim3(256), 0, L, b)
            : launch_kernel(norm_reduce_kernel<T>, dim3(unsigned((a.H + 31) / 32), roles),
                            dim3(1024), 0, L, b);
    if (e != hipSuccess) return e;
    sums.launched = true;
    L.start = nullptr;
    r = stop;
  }
  return hipSuccess;
}

}  // namespace

// Units of one launch: about as many as the chip holds at once (256 CUs x 12 to
// 16 wavefronts, of which a wider row's block takes more), each of at least one
// row.  bf16, post norm (pre norm): H = 2048, 1024 units 77.6 us, 512 76.6, 768
// 77.7; H = 512, 1024 blocks of four 87.4 (61.4), 768 79.6 (61.2), 512 79.0
// (62.9); H = 768, 2048 units 83.4, 1024 90.9.
NormUnits plan_norm_units(int64_t N, int64_t hv, int64_t gate_rows, int64_t gate_span) {
  NormUnits u;
  // units side by side in a block: kSide of the backward's threads per row
  u.blocks_of = hv <= 8 ? 32 : hv <= 16 ? 16 : hv <= 32 ? 8 : hv <= 64 ? 4 : 1;
  if (N <= 0) {  // no units: the sums are of nothing
    u.per_group = u.blocks_of;
    return u;
  }
  const int64_t most = hv <= 64 ? 768 * u.blocks_of : hv <= 128 ? 2048 : hv <= 256 ? 1024
                       : hv <= 512 ? 512 : 256;
  const int64_t rows = (N + most - 1) / most;
  auto whole = [&](int64_t n) { return (n + u.blocks_of - 1) / u.blocks_of * u.blocks_of; };
  // Units of whole groups need no sums for the gate: for groups no longer than a
  // unit (16384 x 2048, 1024 gate rows: 241 -> 47 us), and for enough groups to
  // fill the chip by themselves (512 gate rows: 64 -> 51; 256: 62 -> 73).
  const bool fill = gate_rows >= 512 && gate_rows >= 128 * u.blocks_of;
  if (gate_rows == 1 || (gate_span > rows && !fill)) {
    u.per_group = whole((gate_span + rows - 1) / rows);
    u.rows = rows;
    u.count = gate_rows * u.per_group;
  } else {
    u.per_group = 0;
    u.rows = gate_span > rows ? gate_span : rows / gate_span * gate_span;
    u.count = whole((N + u.rows - 1) / u.rows);
  }
  return u;
}

hipError_t launch_norm_fwd(const NormFwd& a, bool post, bool next, int dtype, const Launch& s) {
  return dtype == TOPMOE_DTYPE_FP32 ? fwd_typed<float>(a, post, next, s)
                                    : fwd_typed<bf16_t>(a, post, next, s);
}

hipError_t launch_norm_bwd(const NormBwd& a, bool post, bool next, int dtype, const Launch& rows,
                           const Launch& sums) {
  return dtype == TOPMOE_DTYPE_FP32 ? bwd_typed<float>(a, post, next, rows, sums)
                                    : bwd_typed<bf16_t>(a, post, next, rows, sums);
}

}  // namespace topmoe
