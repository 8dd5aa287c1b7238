// Products of few grouped rows (gfx950, wave64): the matrix is read once from
// memory straight into the matrix instructions' registers.  Layouts and
// formats: mm.h.
//
// A block takes 16 CT columns of one expert's matrix for all the expert's
// rows, 16 RT of them at a time; its WK wavefronts divide K and add their sums
// through LDS at the end, in a fixed order.  A lane loads 16 bytes of its
// column (or of its row) at a time: 32 k of e2m1, 8 of bf16, 4 of fp32; which k
// a lane group holds does not matter to the sum as long as row and column
// agree.  Nothing is staged: rows are few and come from the caches.  Bound by
// the matrix's bytes (bf16, 64 rows of 16 experts, 2048 -> 1408, in 64 x 64 tiles
// 14 us, 6.5 TB/s) or, where they are few, by one load's way (4-bit, one row, 2048
// -> 6464: 5.3 us for 7 MB; 64 rows of 16 experts, 2048 -> 1408: 11 for 24 MB).
// The launchers take it by the average rows of an expert, which is all the host
// knows; an expert of many more has no more blocks for them, and each reads its
// columns again for every 16 RT rows (us here and in tiles: 64 experts, 2048 ->
// 1408, 8 rows each, bf16 by 4 bits 38 and 86; 64 experts, 768 -> 256, one of 600
// rows and 4 each in the others, bf16 97 and 9, fp32 124 and 30, bf16 by 4 bits 49
// and 11; 256 experts, 768 -> 768, one of 2000 and 1 each, fp32 499 and 184, bf16 by
// 4 bits 171 and 74; 16 experts, 2048 -> 1408, one of 200 and 3 each, 4-bit rows 34
// and 12).
#pragma once

#include "mm_impl.h"

namespace topmoe {
namespace mm {

__device__ __forceinline__ f32x4 mfma16_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16_f32(u32x4 a, u32x4 b, f32x4 c) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[s]), __uint_as_float(b[s]), c, 0, 0,
                                             0);
  return c;
}
template <int FA>  // 0 e4m3, 4 e2m1
__device__ __forceinline__ f32x4 mfma16_mx(u32x4 a0, u32x4 a1, u32x4 b, f32x4 c, uint32_t sa,
                                           uint32_t sb) {
  const i32x8 x = {int(a0[0]), int(a0[1]), int(a0[2]), int(a0[3]),
                   int(a1[0]), int(a1[1]), int(a1[2]), int(a1[3])};
  const i32x8 y = {int(b[0]), int(b[1]), int(b[2]), int(b[3]), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, FA, 4, 0, int(sa), 0, int(sb));
}

// 16-byte pieces of a row's k that meet a lane's 16 bytes of a column.
constexpr int few_pieces(int fa, int fb) {
  return fb != kMmE2m1 && fb != kMmE2m1Bf ? 1
         : fa == kMmE2m1 ? 1 : fa == kMmE4m3 || fa == kMmE4m3Bf ? 2 : fa == kMmBf16 ? 4 : 8;
}

template <int FA, int FB, typename OT, int RT, int CT, int WK>
__global__ __launch_bounds__(64 * WK) void mm_few_kernel(MmParams p) {
  constexpr bool W4 = FB == kMmE2m1 || FB == kMmE2m1Bf, MX = FB == kMmE2m1;
  constexpr bool SA = mm_scaled(FA);
  constexpr int LK = 128 / mm_bits(FB);     // k of a lane's 16 bytes
  constexpr int KS = 4 * LK;                // k of a step
  constexpr int PA = few_pieces(FA, FB);
  constexpr int NS = FA == kMmF32Split ? 3 : 1;
  constexpr int U = W4 ? 2 : 4;             // steps in flight
  constexpr int COLS = 16 * CT, LD = COLS + 4;
  __shared__ float s_sum[WK][16 * RT][LD];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l = lane & 15, g = lane >> 4;
  const int e = blockIdx.y, n0 = blockIdx.x * COLS;
  int begin = 0, end = int(p.R);
  if (p.offsets != nullptr) {
    begin = offset_at(p.offsets, e, p.E, p.R);
    end = e < p.E ? offset_at(p.offsets, e + 1, p.E, p.R) : int(p.R);
  }
  begin = __builtin_amdgcn_readfirstlane(begin);
  end = __builtin_amdgcn_readfirstlane(end);
  if (begin >= end) return;
  OT* out = static_cast<OT*>(p.C);
  if (e == p.E && p.offsets != nullptr) {  // rows of no expert
    for (int64_t i = tid; i < int64_t(end - begin) * (COLS / 4); i += 64 * WK) {
      const int c = n0 + int(i % (COLS / 4)) * 4;
      const float z[4] = {0.f, 0.f, 0.f, 0.f};
      if (c < p.N) store4<OT>(out + (begin + i / (COLS / 4)) * p.ldc + c, z);
    }
    return;
  }
  const int KB = p.K / 32;
  // this wavefront's steps
  const int steps = (p.K + KS - 1) / KS, share = (steps + WK - 1) / WK;
  const int first = wid * share, last = first + share < steps ? first + share : steps;
  const char* bcol[CT];
  const uint8_t* bscale[W4 ? CT : 1];
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    int n = n0 + 16 * j + l;
    n = n < p.N ? n : p.N - 1;  // its sums are not stored
    const int64_t col = int64_t(e) * p.N + n;
    bcol[j] = static_cast<const char*>(p.B) + col * p.K * mm_bits(FB) / 8;
    if constexpr (W4) bscale[j] = p.Bs + col * KB;
  }

  for (int r0 = begin; r0 < end; r0 += 16 * RT) {
    const char* arow[RT];
    const uint8_t* ascale[SA ? RT : 1];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      int r = r0 + 16 * i + l;
      r = r < end ? r : end - 1;
      arow[i] = static_cast<const char*>(p.A) + int64_t(r) * p.lda * mm_bits(FA) / 8;
      if constexpr (SA) ascale[i] = p.As + int64_t(r) * KB;
    }
    f32x4 acc[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // What a lane holds of a step: its 16 bytes of each column and the pieces
    // of each row that meet them, with their scale bytes.
    struct Step {
      u32x4 b[CT], a[RT][PA];
      uint32_t sb[W4 ? CT : 1], sa[SA ? RT : 1];
    };
    auto load = [&](int s, Step& t, auto checked) {
      const int k = s * KS + g * LK;
      const bool in = !decltype(checked)::value || k < p.K;
      const int kk = in ? k : 0;
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        t.b[j] = *reinterpret_cast<const u32x4*>(bcol[j] + int64_t(kk) * mm_bits(FB) / 8);
        if (!in) t.b[j] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (W4) t.sb[j] = in ? bscale[j][kk / 32] : 127u;
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
#pragma unroll
        for (int q = 0; q < PA; ++q) {
          int64_t at = int64_t(kk) * mm_bits(FA) / 8 + 16 * q;
          bool ok = in;
          if constexpr (FA == kMmE4m3) {
            // the 8-bit instruction's order: bytes 16 g of the step's first 64 k, then of its second
            const int b = s * KS + 64 * q + 16 * g;
            ok = !decltype(checked)::value || b < p.K;
            at = ok ? b : 0;
          }
          t.a[i][q] = *reinterpret_cast<const u32x4*>(arow[i] + at);
          if (!ok) t.a[i][q] = u32x4{0u, 0u, 0u, 0u};
        }
        if constexpr (SA) t.sa[i] = in ? ascale[i][kk / 32] : 127u;
      }
    };
    auto use = [&](const Step& t) {
      if constexpr (MX) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < CT; ++j)
            acc[i][j] = mfma16_mx<FA == kMmE4m3 ? 0 : 4>(t.a[i][0], t.a[i][PA - 1], t.b[j],
                                                         acc[i][j], t.sa[i], t.sb[j]);
      } else if constexpr (W4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // 8 k each
          u32x4 w[CT];
#pragma unroll
          for (int j = 0; j < CT; ++j) w[j] = bf16_of_e2m1x8(t.b[j][q], scale_f32(t.sb[j]));
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            u32x4 part[NS];
            if constexpr (FA == kMmF32Split) split3(t.a[i][2 * q], t.a[i][2 * q + 1], part);
            else if constexpr (FA == kMmE4m3Bf)
              part[0] = bf16_of_e4m3x8(t.a[i][q / 2][2 * (q % 2)], t.a[i][q / 2][2 * (q % 2) + 1],
                                       scale_f32(t.sa[i]));
            else part[0] = t.a[i][q];
#pragma unroll
            for (int j = 0; j < CT; ++j)
#pragma unroll
              for (int s = NS - 1; s >= 0; --s)
                acc[i][j] = mfma16_bf16(part[s], w[j], acc[i][j]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < CT; ++j)
            acc[i][j] = FB == kMmF32 ? mfma16_f32(t.a[i][0], t.b[j], acc[i][j])
                                     : mfma16_bf16(t.a[i][0], t.b[j], acc[i][j]);
      }
    };
    // whole steps U at a time; the rest one by one, the last perhaps past K
    const int whole = p.K / KS < last ? p.K / KS : last;
    int s = first;
    for (; s + U <= whole; s += U) {
      Step t[U];
#pragma unroll
      for (int u = 0; u < U; ++u) load(s + u, t[u], std::false_type{});
#pragma unroll
      for (int u = 0; u < U; ++u) use(t[u]);
    }
    for (; s < last; ++s) {
      Step t;
      load(s, t, std::true_type{});
      use(t);
    }

    // lane (l, g), register v: row 4 g + v, column l
    __syncthreads();  // the sums of the rows before have been read
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) s_sum[wid][16 * i + 4 * g + v][16 * j + l] = acc[i][j][v];
    __syncthreads();
    for (int t = tid; t < 16 * RT * (COLS / 4); t += 64 * WK) {
      const int r = t / (COLS / 4), c = t % (COLS / 4) * 4;
      if (r0 + r >= end) break;
      if (n0 + c >= p.N) continue;
      f32x4 sum = *reinterpret_cast<const f32x4*>(&s_sum[0][r][c]);
#pragma unroll
      for (int w = 1; w < WK; ++w) {
        const f32x4 o = *reinterpret_cast<const f32x4*>(&s_sum[w][r][c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += o[i];
      }
      const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
      store4<OT>(out + int64_t(r0 + r) * p.ldc + n0 + c, v);
    }
  }
}

template <int FA, int FB, typename OT, int RT, int CT, int WK>
hipError_t launch_few(const MmParams& p, const Launch& s) {
  const dim3 grid(unsigned((p.N + 16 * CT - 1) / (16 * CT)),
                  unsigned(p.offsets == nullptr ? 1 : p.E + 1));
  return launch_kernel(mm_few_kernel<FA, FB, OT, RT, CT, WK>, grid, dim3(64 * WK), 0, s, p);
}

}  // namespace mm
}  // namespace topmoe
