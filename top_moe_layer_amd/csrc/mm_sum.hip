// Sums of the backward's parts (mm.h), in their order: fp32 partial results of
// chunks of the contracted dimension, rounded once to the dtype.  Bound by
// memory: each part is read once.
#include "mm_impl.h"
#include "vec16.h"

#include "../../include/topmoe.h"

namespace topmoe {

namespace {

template <typename T>
__global__ __launch_bounds__(256) void sum_chunks_kernel(const float* __restrict__ part, int chunks,
                                                         int64_t n4, int64_t N4,
                                                         T* __restrict__ out, int64_t ldo) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n4; i += int64_t(gridDim.x) * 256) {
    const f32x4* p = reinterpret_cast<const f32x4*>(part) + i;
    f32x4 s = p[0];
    for (int c = 1; c < chunks; ++c) {
      const f32x4 v = p[c * n4];
#pragma unroll
      for (int w = 0; w < 4; ++w) s[w] += v[w];
    }
    const float v[4] = {s[0], s[1], s[2], s[3]};
    store4<T>(out + i / N4 * ldo + i % N4 * 4, v);
  }
}

// An expert that has several parts, 1024 elements a block and round.
template <typename T>
__global__ __launch_bounds__(256) void sum_rows_kernel(const float* __restrict__ part,
                                                       const int32_t* __restrict__ offsets, int E,
                                                       int64_t R, int most, int64_t MN,
                                                       T* __restrict__ out) {
  const int lane = threadIdx.x & 63, e = blockIdx.y;
  const int rows = lane < E ? mm::offset_at(offsets, lane + 1, E, R) -
                                  mm::offset_at(offsets, lane, E, R) : 0;
  const int parts = mm::parts_of(rows, most), kept = parts > 1 ? parts : 0;
  const int before = wave_inclusive_scan(kept, lane) - kept;
  const int slot = __builtin_amdgcn_readlane(before, e);
  const int room = int(mm_tn_parts(R, most, E)) - slot;  // all of them, unless offsets do decrease
  int n = __builtin_amdgcn_readlane(kept, e);
  n = n < room ? n : room;
  if (n <= 0) return;
  for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4; i < MN;
       i += int64_t(gridDim.x) * 1024) {
    const float* p = part + slot * MN + i;
    f32x4 s = load_vec<true, f32x4>(p);
    for (int c = 1; c < n; ++c) {
      const f32x4 v = load_vec<true, f32x4>(p + c * MN);
#pragma unroll
      for (int w = 0; w < 4; ++w) s[w] += v[w];
    }
    const float v[4] = {s[0], s[1], s[2], s[3]};
    store4<T>(out + e * MN + i, v);
  }
}

}  // namespace

hipError_t launch_mm_sum_chunks(const float* part, int64_t chunks, int64_t R, int64_t N, int dtype,
                                void* out, int64_t ldo, const Launch& s) {
  const int64_t n4 = R * N / 4;
  const dim3 grid(unsigned((n4 + 255) / 256 < 8192 ? (n4 + 255) / 256 : 8192));
  if (dtype == TOPMOE_DTYPE_FP32)
    return launch_kernel(sum_chunks_kernel<float>, grid, dim3(256), 0, s, part, int(chunks), n4,
                         N / 4, static_cast<float*>(out), ldo);
  return launch_kernel(sum_chunks_kernel<bf16_t>, grid, dim3(256), 0, s, part, int(chunks), n4,
                       N / 4, static_cast<bf16_t*>(out), ldo);
}

hipError_t launch_mm_sum_rows(const MmParams& p, int dtype, const Launch& s) {
  const int64_t MN = int64_t(p.M) * p.N;
  // few enough blocks that those of experts of one part, which end at once, cost little
  const int64_t all = (MN + 1023) / 1024, most = 2048 / p.E;  // E <= 16
  const dim3 grid(unsigned(all < most ? all : most), unsigned(p.E));
  if (dtype == TOPMOE_DTYPE_FP32)
    return launch_kernel(sum_rows_kernel<float>, grid, dim3(256), 0, s, p.part, p.offsets, p.E,
                         p.R, p.most, MN, static_cast<float*>(p.C));
  return launch_kernel(sum_rows_kernel<bf16_t>, grid, dim3(256), 0, s, p.part, p.offsets, p.E, p.R,
                       p.most, MN, static_cast<bf16_t*>(p.C));
}

}  // namespace topmoe
