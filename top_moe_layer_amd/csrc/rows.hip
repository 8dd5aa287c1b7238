// Tokens sorted by expert and back, with their weights, and the gradients:
// the dispatch and combine of a top-k MoE whose experts are the caller's own.
//
// Entry i = t * k + j is token t's slot j with expert idx[i].  Its rank within
// the expert counts the earlier entries of the same expert, so the sort is
// stable; an expert keeps its first `cap` entries (all without a capacity).
// The kept entries' rows come first, grouped by ascending expert; entries not
// kept -- over the capacity, or with idx outside [0, E), as a padding token's
// -- get the rows behind them, by (expert, rank), those without an expert last
// ("bucket" E).  entry -> row is thus a bijection on [0, N k): row, or
// -1 - row for an entry that is not kept, whose row holds zeros.
//
//   dispatch      xs[row(i)] = x[t]            dx[t] = sum_j dxs[row(t, j)]
//   combine       y[t] = residual[t] + sum_j alpha[t, j] ys[row(t, j)]
//   its gradient  dys[row(i)] = alpha[i] dy[t],  dalpha[i] = dy[t] . ys[row(i)]
//
// Sums run over the slots in order, in fp32, and are rounded once.  Everything
// here only moves rows: bound by memory, and at decode sizes by the launches
// (kernels of 3 to 5 us behind about 9 to 12 us of host work).  On an MI355X,
// bf16: dispatch of 16384 x 768, top-2, 17.5 us (4.3 TB/s, see the one-launch
// kernel), back 13 us (5.6 TB/s); combine gradient of 16384 x 2048, k = 2,
// 54 us (6.2 TB/s), all moving no more than each input and output once.
#include "kernels.h"
#include "vec16.h"

#include "../../include/topmoe.h"

namespace topmoe {

namespace {

// Words of a histogram's copies: 32 of them up to 71 experts, 8 at 256.
constexpr int kDispatchHist = 32 * 72;
// Up to so many entries 256 threads count them.
constexpr int kDispatchFew = 1024;

__device__ __forceinline__ int bucket_of(int e, int E) { return e >= 0 && e < E ? e : E; }

// Offsets of the kept rows and of the rows behind them, from the buckets'
// totals in LDS: off[b] = sum of min(tot, cap) before b, tail[b] = all kept
// rows + sum of the entries not kept before b.  One wavefront.
__device__ __forceinline__ void scan_buckets(const int* tot, int E, int cap, int* off, int* tail,
                                             int lane) {
  int kept0 = 0, left0 = 0;
  for (int b0 = 0; b0 <= E; b0 += 64) {
    const int b = b0 + lane;
    const int c = b <= E ? tot[b] : 0;
    const int keep = b >= E ? 0 : (cap < c ? cap : c);
    const int ks = wave_inclusive_scan(keep, lane), ls = wave_inclusive_scan(c - keep, lane);
    if (b <= E) {
      off[b] = kept0 + ks - keep;
      tail[b] = left0 + ls - (c - keep);
    }
    kept0 += __shfl(ks, 63, 64);
    left0 += __shfl(ls, 63, 64);
  }
  for (int b = lane; b <= E; b += 64) tail[b] += kept0;
}

// Row of an entry of bucket b with rank r: the row, or -1 - row if not kept.
__device__ __forceinline__ int row_of(int b, int r, int E, int cap, const int* tot,
                                      const int* off, const int* tail) {
  const int lim = b >= E ? 0 : (cap < tot[b] ? cap : tot[b]);
  return r < lim ? off[b] + r : -1 - (tail[b] + r - lim);
}

// The lanes with the same bucket (of the valid ones), by one ballot per bit of it.
__device__ __forceinline__ uint64_t same_bucket(int b, bool valid, int bits) {
  uint64_t peers = __ballot(valid);
  for (int s = 0; s < bits; ++s) {
    const uint64_t m = __ballot((b >> s) & 1);
    peers &= ((b >> s) & 1) ? m : ~m;
  }
  return peers;
}

// ---- large calls: counts per chunk of entries, rows, then the copy ---------
__global__ __launch_bounds__(256) void dispatch_count_kernel(const int32_t* __restrict__ idx,
                                                             int64_t n, int chunk, int E,
                                                             int32_t* __restrict__ part) {
  __shared__ int hist[kDispatchMaxExperts + 1];
  for (int b = threadIdx.x; b <= E; b += 256) hist[b] = 0;
  __syncthreads();
  const int64_t i0 = int64_t(blockIdx.x) * chunk;
  const int64_t i1 = i0 + chunk < n ? i0 + chunk : n;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += 256) atomicAdd(&hist[bucket_of(idx[i], E)], 1);
  __syncthreads();
  for (int b = threadIdx.x; b <= E; b += 256) part[int64_t(blockIdx.x) * (E + 1) + b] = hist[b];
}

// One block per chunk: every bucket's total and the count in earlier chunks
// from the counts of all chunks, then the rank of each of its entries.  The
// wavefronts take an equal part of the chunk each, 64 entries at a time.
constexpr int kPlaceWaves = 16;  // a chunk is a multiple of 1024 entries

__global__ __launch_bounds__(64 * kPlaceWaves) void dispatch_place_kernel(
    const int32_t* __restrict__ idx, int64_t n, int chunk, int nchunk, int E, int bits, int cap,
    const int32_t* __restrict__ part, int32_t* __restrict__ offsets,
    int32_t* __restrict__ row_entry, int32_t* __restrict__ entry_row) {
  constexpr int NT = 64 * kPlaceWaves;
  __shared__ int tot[kDispatchMaxExperts + 1], off[kDispatchMaxExperts + 1];
  __shared__ int tail[kDispatchMaxExperts + 1];
  __shared__ int run[kPlaceWaves][kDispatchMaxExperts + 1];  // next rank of a wavefront's entries
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int B = E + 1;
  for (int b = tid; b < B; b += NT) tot[b] = tail[b] = 0;
  for (int i = tid; i < kPlaceWaves * (kDispatchMaxExperts + 1); i += NT) (&run[0][0])[i] = 0;
  __syncthreads();
  const int64_t share = chunk / kPlaceWaves;
  const int64_t w0 = int64_t(blockIdx.x) * chunk + wave * share;
  const int64_t w1 = w0 + share < n ? w0 + share : n;
  for (int64_t i = w0 + lane; i < w1; i += 64) atomicAdd(&run[wave][bucket_of(idx[i], E)], 1);
  // totals, and counts before this chunk in tail[] (free until the scan)
  int shift = 0;
  while ((1 << shift) < B && shift < 8) ++shift;  // lanes along a chunk's counts
  const int span = 1 << shift, slices = NT >> shift;
  for (int b = tid & (span - 1); b < B; b += span) {
    int all = 0, before = 0;
    for (int c0 = tid >> shift; c0 < nchunk; c0 += slices * 8) {
      int v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int c = c0 + u * slices;
        v[u] = c < nchunk ? part[int64_t(c) * B + b] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        all += v[u];
        before += c0 + u * slices < int(blockIdx.x) ? v[u] : 0;
      }
    }
    atomicAdd(&tot[b], all);
    atomicAdd(&tail[b], before);
  }
  __syncthreads();
  for (int b = tid; b < B; b += NT) {  // first rank of each wavefront's entries
    int r = tail[b];
    for (int w = 0; w < kPlaceWaves; ++w) {
      const int c = run[w][b];
      run[w][b] = r;
      r += c;
    }
  }
  __syncthreads();
  if (wave == 0) {
    scan_buckets(tot, E, cap, off, tail, lane);
    if (blockIdx.x == 0)
      for (int b = lane; b <= E; b += 64) offsets[b] = off[b];
  }
  __syncthreads();
  const uint64_t lt_mask = lane == 0 ? 0ull : (~0ull >> (64 - lane));
  for (int64_t base = w0; base < w1; base += 64) {
    const int64_t i = base + lane;
    const bool valid = i < w1;
    const int b = valid ? bucket_of(idx[i], E) : 0;
    const uint64_t peers = same_bucket(b, valid, bits);
    if (valid) {
      const int r = row_of(b, run[wave][b] + __popcll(peers & lt_mask), E, cap, tot, off, tail);
      entry_row[i] = r;
      row_entry[r < 0 ? -1 - r : r] = r < 0 ? -1 : int32_t(i);
    }
    __builtin_amdgcn_wave_barrier();
    if (valid && (peers & lt_mask) == 0ull) run[wave][b] += __popcll(peers);
    __builtin_amdgcn_wave_barrier();
  }
}

// Token-major copy: each thread reads one piece of a token's row once and
// writes it to the token's k rows (zeros to the rows of entries not kept).  NT:
// x read non-temporally, from 96 MiB of rows on (with a reader of them: 70.4 ->
// 66.8 us at 96 MiB, 94.9 -> 89.5 at 132; alone 24.5 -> 27.6 at 65).
template <bool NT>
__global__ __launch_bounds__(256) void dispatch_copy_kernel(const u32x4* __restrict__ x,
                                                            const int32_t* __restrict__ entry_row,
                                                            int64_t t0, uint32_t pieces, int hv,
                                                            int k, u32x4* __restrict__ xs) {
  const uint32_t g = blockIdx.x * 256u + threadIdx.x;
  if (g >= pieces) return;
  const uint32_t dt = g / uint32_t(hv), p = g - dt * uint32_t(hv);
  const int64_t t = t0 + dt;
  const u32x4 v = load_piece<NT>(x + t * hv + p);
  for (int j = 0; j < k; ++j) {
    const int r = entry_row[t * k + j];
    if (r >= 0) xs[int64_t(r) * hv + p] = v;
    else xs[int64_t(-1 - r) * hv + p] = u32x4{0u, 0u, 0u, 0u};
  }
}

// ---- up to kDispatchOne entries: one launch ----------------------------------
// Every block counts all n entries itself (n * 4 bytes, from L2) and so knows
// its own entries' rows without waiting for another block.  Counts go to one
// of `copies` histograms by lane (up to 32, as many as the space holds), so
// that the lanes of a wavefront that meet the same expert seldom add to the
// same word.  The first pieces of the block's own tokens are loaded before the
// counting.  A block's own entries (at most kSegs batches of 64) take a
// wavefront a batch: the lanes of one bucket find each other by ballots, and
// each batch's counts give the others their first ranks.  256 blocks of 1024
// threads (256 up to kDispatchFew entries: 32 tokens 4.2 against 5.2 us).  At
// 32768 entries the counting takes about 5.5 us, 33 MB from L2 on all CUs, and
// the rows' loads run under it; one copy of the histogram instead of 32 costs
// another 5 us, 8 or 64 nothing.
template <int NT>
__global__ __launch_bounds__(NT) void dispatch_one_kernel(
    const u32x4* __restrict__ x, const int32_t* __restrict__ idx, int n, int N, int tb, int hv,
    int E, int k, int bits, int copies, int cap, u32x4* __restrict__ xs,
    int32_t* __restrict__ offsets, int32_t* __restrict__ row_entry,
    int32_t* __restrict__ entry_row) {
  constexpr int kPre = NT == 1024 ? 6 : 2, kIn = NT == 1024 ? 32 : 4;  // in flight per thread:
                                                                       // pieces, entries
  constexpr int kMost = NT == 1024 ? kDispatchOne : kDispatchFew;
  constexpr int kOwn = kMost / 256 + kDispatchMaxExperts;  // tb * k <= n / 256 + k
  constexpr int kWaves = NT / 64, kSegs = (kOwn + 63) / 64, kTurns = (kSegs + kWaves - 1) / kWaves;
  __shared__ int hist[2][kDispatchHist];  // [copies][B]: entries before the block's, from it on
  __shared__ int tot[kDispatchMaxExperts + 1], before[kDispatchMaxExperts + 1];
  __shared__ int off[kDispatchMaxExperts + 1], tail[kDispatchMaxExperts + 1];
  __shared__ int seg[kSegs][kDispatchMaxExperts + 1];
  __shared__ int rows[kOwn];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int B = E + 1;
  const int t0 = blockIdx.x * tb, t1 = t0 + tb < N ? t0 + tb : N;
  const int e0 = t0 * k, own = (t1 - t0) * k;
  const int segs = (own + 63) / 64;
  const int pieces = (t1 - t0) * hv;
  const u32x4* xb = x + int64_t(t0) * hv;  // the block's rows are consecutive
  int ex[kTurns];  // this wavefront's own entries
#pragma unroll
  for (int q = 0; q < kTurns; ++q) {
    const int i = (q * kWaves + wave) * 64 + lane;
    ex[q] = i < own ? idx[e0 + i] : 0;
  }
  u32x4 pre[kPre];
#pragma unroll
  for (int u = 0; u < kPre; ++u) {
    const int p = tid + u * NT;
    pre[u] = load_piece_if(p < pieces, xb + p);
  }
  for (int i = tid; i < copies * B; i += NT) hist[0][i] = hist[1][i] = 0;
  for (int i = tid; i < segs * (kDispatchMaxExperts + 1); i += NT) (&seg[0][0])[i] = 0;
  __syncthreads();
  const uint64_t lt_mask = lane == 0 ? 0ull : (~0ull >> (64 - lane));
  int rank[kTurns];  // within the batch
#pragma unroll
  for (int q = 0; q < kTurns; ++q) {
    const int w = q * kWaves + wave;
    const bool valid = w * 64 + lane < own;
    const int b = valid ? bucket_of(ex[q], E) : 0;
    const uint64_t peers = same_bucket(b, valid, bits);
    rank[q] = __popcll(peers & lt_mask);
    if (valid && rank[q] == 0) seg[w][b] = __popcll(peers);
  }
  const int mine = (lane & (copies - 1)) * B;
  for (int i0 = tid; i0 < n; i0 += NT * kIn) {
    int e[kIn];
#pragma unroll
    for (int u = 0; u < kIn; ++u) e[u] = i0 + u * NT < n ? idx[i0 + u * NT] : 0;
#pragma unroll
    for (int u = 0; u < kIn; ++u) {
      const int i = i0 + u * NT;
      if (i < n) atomicAdd(&hist[i < e0 ? 0 : 1][mine + bucket_of(e[u], E)], 1);
    }
  }
  __syncthreads();
  for (int b = tid; b < B; b += NT) {
    int pre_b = 0, from_b = 0;
    for (int c = 0; c < copies; ++c) {
      pre_b += hist[0][c * B + b];
      from_b += hist[1][c * B + b];
    }
    before[b] = pre_b;
    tot[b] = pre_b + from_b;
  }
  __syncthreads();
  if (wave == 0) {
    scan_buckets(tot, E, cap, off, tail, lane);
    if (blockIdx.x == 0)
      for (int b = lane; b <= E; b += 64) offsets[b] = off[b];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kTurns; ++q) {
    const int w = q * kWaves + wave, i = w * 64 + lane;
    if (i < own) {
      const int b = bucket_of(ex[q], E);
      int first = before[b];
      for (int v = 0; v < w; ++v) first += seg[v][b];
      const int r = row_of(b, first + rank[q], E, cap, tot, off, tail);
      rows[i] = r;
      entry_row[e0 + i] = r;
      row_entry[r < 0 ? -1 - r : r] = r < 0 ? -1 : e0 + i;
    }
  }
  __syncthreads();
  auto put = [&](int g, u32x4 v) {
    const int t = g / hv, p = g - t * hv;
    for (int j = 0; j < k; ++j) {
      const int r = rows[t * k + j];
      if (r >= 0) xs[int64_t(r) * hv + p] = v;
      else xs[int64_t(-1 - r) * hv + p] = u32x4{0u, 0u, 0u, 0u};
    }
  };
#pragma unroll
  for (int u = 0; u < kPre; ++u)
    if (tid + u * NT < pieces) put(tid + u * NT, pre[u]);
  for (int g = tid + kPre * NT; g < pieces; g += NT) put(g, load_piece(xb + g));
}

__global__ void dispatch_empty_kernel(int E, int32_t* offsets) {
  for (int b = threadIdx.x; b <= E; b += 256) offsets[b] = 0;
}

// ---- back to tokens ---------------------------------------------------------
// out[t] = residual[t] (or 0) + sum_j w[t, j] rows[entry_row[t, j]], the
// combine (w = alpha) and the dispatch's gradient (w = 1).  A row id outside
// [0, nrows) adds nothing.  Four slots' pieces are in flight at a time.  NT:
// rows read non-temporally, from 192 MiB of them on (just written, top-2, H =
// 768: 155.5 -> 149.9 us with their writer at 192 MiB, 106.5 -> 108.8 at 132).
template <typename T, bool WEIGHTED, bool NT>
__global__ __launch_bounds__(256) void gather_sum_kernel(
    const T* __restrict__ rows, const int32_t* __restrict__ entry_row,
    const float* __restrict__ alpha, const T* residual, int64_t nrows, int64_t t0,
    uint32_t pieces, int hv, int H, int k, T* out) {
  constexpr int E = kE<T>;
  const uint32_t g = blockIdx.x * 256u + threadIdx.x;
  if (g >= pieces) return;
  const uint32_t dt = g / uint32_t(hv);
  const int64_t t = t0 + dt;
  const int64_t h = int64_t(g - dt * uint32_t(hv)) * E;
  float acc[E];
  unpack(load_piece_if(residual != nullptr, residual + t * H + h), acc);
  const int32_t* er = entry_row + t * k;
  for (int j0 = 0; j0 < k; j0 += 4) {
    u32x4 v[4];
    float w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t r = j0 + u < k ? int64_t(er[j0 + u]) : -1;
      const bool use = r >= 0 && r < nrows;
      w[u] = !use ? 0.f : WEIGHTED ? alpha[t * k + j0 + u] : 1.f;
      v[u] = load_piece_if<NT>(use, rows + r * H + h);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float f[E];
      unpack(v[u], f);
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] = WEIGHTED ? fmaf(w[u], f[i], acc[i]) : acc[i] + f[i];
    }
  }
  store_piece(out + t * H + h, acc);
}

// dys[row(i)] = alpha[i] dy[t] and dalpha[i] = dy[t] . ys[row(i)]: a wavefront,
// or for rows of few pieces a part of one, R lanes per entry, consecutive
// entries in a block, so that a token's k entries share its dy row in the
// caches; each row of ys is read once, non-temporally, and dys written so when
// it is large (NT): 16384 x 2048 bf16, k = 2: 66.3 -> 63.2 -> 54.0 us, 6.2 TB/s.
// Fewer lanes: 32768 tokens, k = 8, H = 64, 128, 256: 71, 78, 89 -> 24, 28, 57 us.
template <typename T, bool NT, int R>
__global__ __launch_bounds__(256) void combine_bwd_kernel(
    const T* __restrict__ dy, const T* __restrict__ ys, const int32_t* __restrict__ entry_row,
    const float* __restrict__ alpha, int64_t n, int64_t i0, int hv, int H, int k,
    T* __restrict__ dys, float* __restrict__ dalpha) {
  const int lane = int(threadIdx.x) % R;
  const int64_t i = i0 + int64_t(blockIdx.x) * (256 / R) + int(threadIdx.x) / R;
  if (i >= n) return;
  const int64_t r = entry_row[i];
  const int64_t row = r < 0 ? -1 - r : r;
  if (row >= n) {  // not a row of this call
    if (lane == 0) dalpha[i] = 0.f;
    return;
  }
  T* o = dys + row * H;
  if (r < 0) {
    for (int p = lane; p < hv; p += R)
      *reinterpret_cast<u32x4*>(o + p * kE<T>) = u32x4{0u, 0u, 0u, 0u};
    if (lane == 0) dalpha[i] = 0.f;
    return;
  }
  const T* d = dy + (i / k) * H;
  const T* s = ys + row * H;
  const float a = alpha[i];
  float dot = 0.f;
  for (int p = lane; p < hv; p += R) {
    float fd[kE<T>], fs[kE<T>];
    unpack(load_piece(d + p * kE<T>), fd);
    unpack(load_piece<true>(s + p * kE<T>), fs);
#pragma unroll
    for (int c = 0; c < kE<T>; ++c) {
      dot = fmaf(fd[c], fs[c], dot);
      fd[c] *= a;
    }
    store_piece<NT>(o + p * kE<T>, fd);
  }
#pragma unroll
  for (int o = R / 2; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
  if (lane == 0) dalpha[i] = dot;
}

// Tokens of one launch: at most 2^30 pieces, so that piece numbers stay in 32
// bits and a grid within its limit of threads.
int64_t slab_rows(int hv) {
  const int64_t m = (int64_t(1) << 30) / hv;
  return m > 0 ? m : 1;
}

template <typename F>
hipError_t for_slabs(int64_t N, int64_t slab, const Launch& L, F launch) {
  for (int64_t t0 = 0; t0 < N; t0 += slab) {
    Launch one = L;
    if (t0 > 0) one.start = nullptr;
    if (t0 + slab < N) one.stop = nullptr;
    const hipError_t e = launch(t0, t0 + slab < N ? slab : N - t0, one);
    if (e != hipSuccess) return e;
    L.launched = true;
  }
  return hipSuccess;
}

hipError_t dispatch_one(const u32x4* x, const int32_t* idx, int64_t N, int hv, int E, int k,
                        int bits, int cap, u32x4* xs, int32_t* offsets, int32_t* row_entry,
                        int32_t* entry_row, const Launch& s) {
  const int tb = int((N + 255) / 256);
  int copies = N * k <= kDispatchFew ? 4 : 32;
  while (copies * (E + 1) > kDispatchHist) copies /= 2;
  const dim3 grid(unsigned((N + tb - 1) / tb));
#define TOPMOE_LAUNCH_ONE(NT)                                                                    \
  return launch_kernel(dispatch_one_kernel<NT>, grid, dim3(NT), 0, s, x, idx, int(N * k), int(N), \
                       tb, hv, E, k, bits, copies, cap, xs, offsets, row_entry, entry_row)
  if (N * k <= kDispatchFew) TOPMOE_LAUNCH_ONE(256);
  TOPMOE_LAUNCH_ONE(1024);
#undef TOPMOE_LAUNCH_ONE
}

hipError_t dispatch_copy(const u32x4* x, const int32_t* entry_row, int64_t N, int hv, int k,
                         u32x4* xs, const Launch& s) {
  return for_slabs(N, slab_rows(hv), s, [&](int64_t t0, int64_t rows, const Launch& L) {
    const uint32_t pieces = uint32_t(rows * hv);
    const auto kernel = N * k * hv * 16 >= kNtBytes / 4 * 3 ? dispatch_copy_kernel<true>
                                                            : dispatch_copy_kernel<false>;
    return launch_kernel(kernel, dim3((pieces + 255) / 256), dim3(256), 0, L, x, entry_row, t0,
                         pieces, hv, k, xs);
  });
}

template <typename T, bool WEIGHTED>
hipError_t gather_sum(const void* rows, const int32_t* entry_row, const float* alpha,
                      const void* residual, int64_t N, int H, int k, void* out,
                      const Launch& s) {
  const int hv = H / kE<T>;
  return for_slabs(N, slab_rows(hv), s, [&](int64_t t0, int64_t m, const Launch& L) {
    const uint32_t pieces = uint32_t(m * hv);
    const auto kernel = N * k * H * int64_t(sizeof(T)) >= kNtBytes / 2 * 3
                            ? gather_sum_kernel<T, WEIGHTED, true>
                            : gather_sum_kernel<T, WEIGHTED, false>;
    return launch_kernel(kernel, dim3((pieces + 255) / 256), dim3(256), 0,
                         L, static_cast<const T*>(rows), entry_row, alpha,
                         static_cast<const T*>(residual), N * k, t0, pieces, hv, H, k,
                         static_cast<T*>(out));
  });
}

template <typename T, int R>
hipError_t combine_bwd(const void* dy, const void* ys, const int32_t* entry_row,
                       const float* alpha, int64_t N, int H, int k, void* dys, float* dalpha,
                       const Launch& s) {
  const int64_t n = N * k;
  return for_slabs(n, int64_t(1) << 24, s, [&](int64_t i0, int64_t m, const Launch& L) {
    const auto kernel = n * H * int64_t(sizeof(T)) >= kNtBytes ? combine_bwd_kernel<T, true, R>
                                                               : combine_bwd_kernel<T, false, R>;
    constexpr int side = 256 / R;
    return launch_kernel(kernel, dim3(unsigned((m + side - 1) / side)), dim3(256), 0, L,
                         static_cast<const T*>(dy), static_cast<const T*>(ys), entry_row, alpha,
                         n, i0, H / kE<T>, H, k, static_cast<T*>(dys), dalpha);
  });
}

}  // namespace

DispatchPlan plan_dispatch(int64_t n, int E) {
  DispatchPlan p;
  if (n <= 0) return p;
  const int64_t c = (n + 255) / 256;  // at most 256 chunks
  p.chunk = int((c + 1023) / 1024 * 1024);
  p.nchunk = int((n + p.chunk - 1) / p.chunk);
  p.bytes = size_t(p.nchunk) * (E + 1) * sizeof(int32_t);
  return p;
}

hipError_t launch_dispatch_rows(const void* x, const int32_t* idx, int64_t N, int H, int E, int k,
                                int cap, int dtype, void* xs, int32_t* offsets,
                                int32_t* row_entry, int32_t* entry_row, int32_t* part,
                                const Launch& rows, const Launch& copy) {
  const int64_t n = N * k;
  const DispatchPlan p = plan_dispatch(n, E);
  if (n == 0) return launch_kernel(dispatch_empty_kernel, dim3(1), dim3(256), 0, rows, E, offsets);
  int bits = 0;
  while ((E >> bits) != 0) ++bits;
  // rows only move: pieces of 16 bytes whatever the type
  const int hv = H / (dtype == TOPMOE_DTYPE_FP32 ? 4 : 8);
  const u32x4* xp = static_cast<const u32x4*>(x);
  u32x4* op = static_cast<u32x4*>(xs);
  if (dispatch_in_one(N, H, k, dtype == TOPMOE_DTYPE_FP32 ? 4 : 2))
    return dispatch_one(xp, idx, N, hv, E, k, bits, cap, op, offsets, row_entry, entry_row, copy);
  Launch first = rows, second = rows;
  first.stop = nullptr;
  second.start = nullptr;
  hipError_t e = launch_kernel(dispatch_count_kernel, dim3(p.nchunk), dim3(256), 0, first, idx, n,
                               p.chunk, E, part);
  if (e != hipSuccess) return e;
  e = launch_kernel(dispatch_place_kernel, dim3(p.nchunk), dim3(64 * kPlaceWaves), 0, second, idx, n, p.chunk,
                    p.nchunk, E, bits, cap, part, offsets, row_entry, entry_row);
  if (e != hipSuccess) return e;
  rows.launched = true;
  return dispatch_copy(xp, entry_row, N, hv, k, op, copy);
}

hipError_t launch_gather_sum(const void* rows, const int32_t* entry_row, const float* alpha,
                             const void* residual, int64_t N, int H, int k, int dtype, void* out,
                             const Launch& s) {
  if (dtype == TOPMOE_DTYPE_FP32)
    return alpha ? gather_sum<float, true>(rows, entry_row, alpha, residual, N, H, k, out, s)
                 : gather_sum<float, false>(rows, entry_row, alpha, residual, N, H, k, out, s);
  return alpha ? gather_sum<bf16_t, true>(rows, entry_row, alpha, residual, N, H, k, out, s)
               : gather_sum<bf16_t, false>(rows, entry_row, alpha, residual, N, H, k, out, s);
}

hipError_t launch_moe_combine_bwd(const void* dy, const void* ys, const int32_t* entry_row,
                                  const float* alpha, int64_t N, int H, int k, int dtype,
                                  void* dys, float* dalpha, const Launch& s) {
#define TOPMOE_COMBINE_BWD(T, R) \
  return combine_bwd<T, R>(dy, ys, entry_row, alpha, N, H, k, dys, dalpha, s)
  if (dtype == TOPMOE_DTYPE_FP32) {
    if (H <= 64) TOPMOE_COMBINE_BWD(float, 16);
    if (H <= 128) TOPMOE_COMBINE_BWD(float, 32);
    TOPMOE_COMBINE_BWD(float, 64);
  }
  if (H <= 128) TOPMOE_COMBINE_BWD(bf16_t, 16);
  if (H <= 256) TOPMOE_COMBINE_BWD(bf16_t, 32);
  TOPMOE_COMBINE_BWD(bf16_t, 64);
#undef TOPMOE_COMBINE_BWD
}

}  // namespace topmoe
