// C ABI entry points of the products of rows grouped by expert and of the
// 4-bit matrices.  See include/topmoe.h for the contract of every function.
#include <stdint.h>

#include "api_util.h"
#include "mm.h"
#include "plan.h"

#include "../../include/topmoe.h"

using namespace topmoe;

static_assert(kMmMaxExperts == TOPMOE_LINEAR_MAX_EXPERTS, "expert limit");
static_assert(kMx4Group == TOPMOE_MX4_GROUP && kMx4Group == kAct8Group, "scale group");

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
// The products', so that a row past a tile's or a slice's last still counts in 32 bits.
constexpr int64_t kMaxLinearRows = (int64_t(1) << 31) - (int64_t(1) << 16);
constexpr int64_t kMaxSide = int64_t(1) << 20, kMaxPitch = int64_t(1) << 21;
// Rows of all experts' matrices: what a launch's threads number in 32 bits.
constexpr int64_t kMaxOut = int64_t(1) << 25;

bool known_dtype(int dtype) {
  return dtype == TOPMOE_DTYPE_FP32 || dtype == TOPMOE_DTYPE_BF16;
}
bool pitch_ok(int64_t ld, int64_t C) { return ld >= C && ld % 8 == 0 && ld <= kMaxPitch; }

// K in, O out; step: what K is a multiple of.
int linear_shape(int64_t R, int64_t K, int64_t O, int E, const int32_t* offsets, int step) {
  if (R < 0 || R > kMaxLinearRows || K <= 0 || K % step != 0 || K > kMaxSide) return TOPMOE_ERR_BAD_SHAPE;
  if (O <= 0 || O % 8 != 0 || O > kMaxSide) return TOPMOE_ERR_BAD_SHAPE;
  if (E < 1 || E > kMmMaxExperts || (!offsets && E != 1)) return TOPMOE_ERR_BAD_SHAPE;
  if (int64_t(E) * O > kMaxOut) return TOPMOE_ERR_BAD_SHAPE;
  return TOPMOE_OK;
}

MmParams params(const void* A, int64_t lda, const void* B, const int32_t* offsets, int64_t R,
                int64_t K, int64_t N, int E, void* C, int64_t ldc) {
  MmParams p{};
  p.A = A; p.lda = lda; p.B = B; p.offsets = offsets; p.R = R; p.K = int(K); p.N = int(N); p.E = E;
  p.C = C; p.ldc = ldc;
  return p;
}

// Two launches of one stage.
void in_one(const Launch& L, Launch* first, Launch* second) {
  *first = L;
  *second = L;
  first->stop = second->start = nullptr;
}

// dx of moe_linear_bwd, with the matrices as they are, or of mx4_linear_bwd, with
// them in bf16 (by_bf16); `part`: for the sums in parts.
hipError_t rows_grad(MmParams p, int dtype, bool by_bf16, float* part, const Launch& L) {
  const bool f32 = dtype == TOPMOE_DTYPE_FP32;
  auto product = [&](const MmParams& q, const Launch& s, bool parts) {
    if (f32) return by_bf16 ? launch_mm_f32_by_bf16(q, s) : launch_mm_f32(kMmNN, q, s);
    return parts ? launch_mm_bf16_parts(q, s) : launch_mm_bf16(kMmNN, q, s);
  };
  p.kchunk = mm_nn_chunk(p.R, p.N, p.K, p.E);
  if (p.kchunk == 0) return product(p, L, false);
  Launch first, second;
  in_one(L, &first, &second);
  MmParams q = p;
  q.C = part;
  q.ldc = p.N;
  const hipError_t e = product(q, first, true);
  if (e != hipSuccess) return e;
  L.launched = true;
  return launch_mm_sum_chunks(part, mm_chunks(p.K, p.kchunk), p.R, p.N, dtype, p.C, p.ldc, second);
}
size_t rows_grad_bytes(int64_t R, int64_t K, int64_t O, int E) {
  const int kchunk = mm_nn_chunk(R, K, O, E);
  return kchunk > 0 ? size_t(mm_chunks(O, kchunk)) * size_t(R) * size_t(K) * sizeof(float) : 0;
}

int mx4_shape(int64_t R, int64_t C) {
  if (R < 0 || R > kMaxRows || C <= 0 || C % 8 != 0 || C > kMaxRows) return TOPMOE_ERR_BAD_SHAPE;
  return TOPMOE_OK;
}
bool mx4_pitch_ok(int64_t ld, int64_t C) { return ld >= C && ld % 8 == 0; }

}  // namespace

extern "C" {

int moe_linear_fwd(const void* x, int64_t ldx, const void* w, const int32_t* expert_offsets,
                   int64_t R, int64_t K, int64_t O, int E, int dtype, void* y, int64_t ldy,
                   void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = linear_shape(R, K, O, E, expert_offsets, 8);
  if (status != TOPMOE_OK) return status;
  if (!pitch_ok(ldx, K) || !pitch_ok(ldy, O)) return TOPMOE_ERR_BAD_SHAPE;
  if (!w || (R > 0 && (!x || !y))) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(expert_offsets, 4))
    return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  const MmParams p = params(x, ldx, w, expert_offsets, R, K, O, E, y, ldy);
  if (R > 0)
    TOPMOE_TRY(dtype == TOPMOE_DTYPE_FP32 ? launch_mm_f32(kMmNT, p, L) : launch_mm_bf16(kMmNT, p, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

size_t moe_linear_bwd_dtype_workspace_bytes(int64_t R, int64_t K, int64_t O, int E, int dtype) {
  int32_t any = 0;
  if (!known_dtype(dtype) || linear_shape(R, K, O, E, &any, 8) != TOPMOE_OK) return 0;
  const size_t dx = rows_grad_bytes(R, K, O, E);
  const int64_t parts =
      mm_tn_parts(R, mm_tn_most(R, O, K, E, dtype == TOPMOE_DTYPE_FP32), E);
  const size_t dw = size_t(parts) * size_t(O) * size_t(K) * sizeof(float);
  return align_up((dx > dw ? dx : dw) + 1);
}

size_t moe_linear_bwd_workspace_bytes(int64_t R, int64_t K, int64_t O, int E) {
  const size_t f32 = moe_linear_bwd_dtype_workspace_bytes(R, K, O, E, TOPMOE_DTYPE_FP32);
  const size_t bf16 = moe_linear_bwd_dtype_workspace_bytes(R, K, O, E, TOPMOE_DTYPE_BF16);
  return f32 > bf16 ? f32 : bf16;
}

int moe_linear_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
                   const int32_t* expert_offsets, int64_t R, int64_t K, int64_t O, int E,
                   int dtype, void* dx, int64_t lddx, void* dw, void* workspace,
                   size_t workspace_bytes, void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = linear_shape(R, K, O, E, expert_offsets, 8);
  if (status != TOPMOE_OK) return status;
  if (!pitch_ok(lddy, O) || (dw && !pitch_ok(ldx, K)) || (dx && !pitch_ok(lddx, K)))
    return TOPMOE_ERR_BAD_SHAPE;
  if ((!dx && !dw && R > 0) || (dx && !w) || !workspace || (R > 0 && (!dy || (dw && !x))))
    return TOPMOE_ERR_NULL_ARG;
  if (workspace_bytes < moe_linear_bwd_dtype_workspace_bytes(R, K, O, E, dtype))
    return TOPMOE_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(dx, 16) ||
      !aligned(dw, 16) || !aligned(expert_offsets, 4) || !aligned(workspace, 256))
    return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch rows = st.at(0), weights = st.at(1);
  const bool f32 = dtype == TOPMOE_DTYPE_FP32;
  float* part = static_cast<float*>(workspace);
  if (dx && R > 0)
    TOPMOE_TRY(rows_grad(params(dy, lddy, w, expert_offsets, R, O, K, E, dx, lddx), dtype, false,
                         part, rows));
  if (dw) {
    MmParams p = params(dy, lddy, x, expert_offsets, R, 0, K, E, dw, K);
    p.M = int(O);
    p.ldb = ldx;
    p.most = mm_tn_most(R, O, K, E, f32);
    p.part = part;
    Launch first = weights, second = weights;
    if (p.most > 0) in_one(weights, &first, &second);
    TOPMOE_TRY(f32 ? launch_mm_f32(kMmTN, p, first) : launch_mm_bf16(kMmTN, p, first));
    weights.launched = true;
    if (p.most > 0) TOPMOE_TRY(launch_mm_sum_rows(p, dtype, second));
  }
  TOPMOE_TRY(st.close(rows));
  TOPMOE_TRY(st.close(weights));
  return TOPMOE_OK;
}

int mx4_pack(const void* x, int64_t ldx, int64_t R, int64_t C, int dtype, uint8_t* q,
             uint8_t* scale, void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = mx4_shape(R, C);
  if (status != TOPMOE_OK) return status;
  if (!mx4_pitch_ok(ldx, C)) return TOPMOE_ERR_BAD_SHAPE;
  if (R > 0 && (!x || !q || !scale)) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(x, 16) || !aligned(q, 4)) return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_mx4_pack(x, ldx, R, C, dtype, q, scale, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

int mx4_unpack(const uint8_t* q, const uint8_t* scale, int64_t R, int64_t C, int dtype, void* x,
               int64_t ldx, void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = mx4_shape(R, C);
  if (status != TOPMOE_OK) return status;
  if (!mx4_pitch_ok(ldx, C)) return TOPMOE_ERR_BAD_SHAPE;
  if (R > 0 && (!x || !q || !scale)) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(x, 16) || !aligned(q, 4)) return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_mx4_unpack(q, scale, R, C, dtype, x, ldx, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

int mx4_linear_fwd(const void* x, int64_t ldx, const uint8_t* x_scale, int rows,
                   const uint8_t* wq, const uint8_t* w_scale, const int32_t* expert_offsets,
                   int64_t R, int64_t K, int64_t O, int E, int dtype, void* y, int64_t ldy,
                   void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  if (rows != TOPMOE_ROWS_PLAIN && rows != TOPMOE_ROWS_ACT8 && rows != TOPMOE_ROWS_MX4)
    return TOPMOE_ERR_BAD_ARG;
  const bool plain = rows == TOPMOE_ROWS_PLAIN;
  const int status = linear_shape(R, K, O, E, expert_offsets, kMx4Group);
  if (status != TOPMOE_OK) return status;
  if (!pitch_ok(plain ? ldx : K, K) || !pitch_ok(ldy, O)) return TOPMOE_ERR_BAD_SHAPE;
  if (!wq || !w_scale || (R > 0 && (!x || !y || (!plain && !x_scale)))) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(x, 16) || !aligned(wq, 16) || !aligned(y, 16) || !aligned(expert_offsets, 4))
    return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  MmParams p = params(x, plain ? ldx : K, wq, expert_offsets, R, K, O, E, y, ldy);
  p.As = plain ? nullptr : x_scale;
  p.Bs = w_scale;
  const bool bf16 = dtype == TOPMOE_DTYPE_BF16;
  // The 8-bit instructions add eight consecutive products at a time and cut each
  // toward zero to a multiple of 2^-13 of 2^(ea + eb), the largest sum of two
  // factors' exponents (a factor 0.5 of the matrix counts as 1 there): less than
  // 2^-12 of the largest product is lost of each, and nothing of the groups' sums.
  // They are taken where y is bf16, at 1.5 times the rate of bf16 instructions
  // (mm_mx4.hip): with one channel in 64 ten times the others, y [32768, 4864] of
  // 768 products each differs from that of whole sums by 1.7e-4 in the norm, a
  // tenth of its rounding; where outliers cancel it can be more than the rounding.
  // For y in fp32 the 8-bit rows go through bf16, which loses nothing between
  // scale bytes 3 and 246.
  const int fa = plain ? (bf16 ? kMmBf16 : kMmF32Split)
                       : rows == TOPMOE_ROWS_MX4 ? kMmE2m1 : bf16 ? kMmE4m3 : kMmE4m3Bf;
  if (R > 0) TOPMOE_TRY(launch_mm_mx4(fa, bf16, p, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

size_t mx4_linear_bwd_workspace_bytes(int64_t R, int64_t K, int64_t O, int E) {
  int32_t any = 0;
  if (linear_shape(R, K, O, E, &any, kMx4Group) != TOPMOE_OK) return 0;
  return align_up(size_t(E) * size_t(O) * size_t(K) * 2) + align_up(rows_grad_bytes(R, K, O, E));
}

int mx4_linear_bwd(const void* dy, int64_t lddy, const uint8_t* wq, const uint8_t* w_scale,
                   const int32_t* expert_offsets, int64_t R, int64_t K, int64_t O, int E,
                   int dtype, void* dx, int64_t lddx, void* workspace, size_t workspace_bytes,
                   void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = linear_shape(R, K, O, E, expert_offsets, kMx4Group);
  if (status != TOPMOE_OK) return status;
  if (!pitch_ok(lddy, O) || !pitch_ok(lddx, K))
    return TOPMOE_ERR_BAD_SHAPE;
  if (!wq || !w_scale || !workspace || (R > 0 && (!dy || !dx))) return TOPMOE_ERR_NULL_ARG;
  if (workspace_bytes < mx4_linear_bwd_workspace_bytes(R, K, O, E))
    return TOPMOE_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(dy, 16) || !aligned(wq, 16) || !aligned(dx, 16) || !aligned(expert_offsets, 4) ||
      !aligned(workspace, 256))
    return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch unpack = st.at(0), product = st.at(1);
  if (R > 0) {
    TOPMOE_TRY(launch_mx4_unpack(wq, w_scale, int64_t(E) * O, K, TOPMOE_DTYPE_BF16, workspace, K,
                                 unpack));
    char* part = static_cast<char*>(workspace) + align_up(size_t(E) * size_t(O) * size_t(K) * 2);
    TOPMOE_TRY(rows_grad(params(dy, lddy, workspace, expert_offsets, R, O, K, E, dx, lddx), dtype,
                         true, reinterpret_cast<float*>(part), product));
  }
  TOPMOE_TRY(st.close(unpack));
  TOPMOE_TRY(st.close(product));
  return TOPMOE_OK;
}

}  // extern "C"
