// C ABI entry points of the operators around an FFN / MoE block: rows by
// expert and back, norms with gate and residual, activations in 8 bits.  See
// include/topmoe.h for the contract of every function.
#include <stdint.h>

#include "api_util.h"
#include "kernels.h"
#include "plan.h"

#include "../../include/topmoe.h"

using namespace topmoe;

static_assert(kDispatchMaxExperts == TOPMOE_DISPATCH_MAX_EXPERTS, "expert limit");
static_assert(kDispatchOne == TOPMOE_DISPATCH_ONE &&
                  kDispatchOneBytes == TOPMOE_DISPATCH_ONE_BYTES,
              "one-launch limits");
static_assert(kAct8Group == TOPMOE_ACT8_GROUP, "scale group");
static_assert(kGateNone == TOPMOE_GATE_NONE && kGateChannel == TOPMOE_GATE_CHANNEL &&
                  kGateToken == TOPMOE_GATE_TOKEN,
              "gate modes");

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

bool known_dtype(int dtype) {
  return dtype == TOPMOE_DTYPE_FP32 || dtype == TOPMOE_DTYPE_BF16;
}

// ---- rows by expert
int rows_shape(int64_t N, int64_t H, int k) {
  if (N < 0 || k < 1 || k > kDispatchMaxExperts || N > kMaxRows / k) return TOPMOE_ERR_BAD_SHAPE;
  if (H <= 0 || H % 8 != 0 || H > (int64_t(1) << 20)) return TOPMOE_ERR_BAD_SHAPE;
  return TOPMOE_OK;
}

// Entries an expert keeps, INT32_MAX = all, -1 = no such capacity: of a factor
// ceil(factor * N * k / E), of the float's own value, or the capacity itself.
int kept_entries(float factor, int64_t N, int k, int E) {
  if (!nonneg_finite(factor)) return -1;
  if (factor == 0.f) return INT32_MAX;
  const double c = ceil(double(factor) * double(N) * double(k) / double(E));
  return c >= double(N) * double(k) ? INT32_MAX : int(c);
}
int kept_entries(int64_t capacity, int64_t, int, int) {
  return capacity < 0 ? -1 : capacity == 0 || capacity > kMaxRows ? INT32_MAX : int(capacity);
}

template <typename Capacity>
int dispatch_fwd(const void* x, const int32_t* topk_idx, int64_t N, int64_t H, int E, int k,
                 Capacity capacity, int dtype, void* xs, int32_t* expert_offsets,
                 int32_t* row_entry, int32_t* entry_row, void* workspace, size_t workspace_bytes,
                 void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  if (E < 1 || E > kDispatchMaxExperts || k > E) return TOPMOE_ERR_BAD_SHAPE;
  const int status = rows_shape(N, H, k);
  if (status != TOPMOE_OK) return status;
  const bool one = dispatch_in_one(N, H, k, dtype == TOPMOE_DTYPE_FP32 ? 4 : 2);
  const size_t need = one ? 0 : plan_dispatch(N * k, E).bytes;
  if (!expert_offsets || (need > 0 && !workspace) ||
      (N > 0 && (!x || !topk_idx || !xs || !row_entry || !entry_row)))
    return TOPMOE_ERR_NULL_ARG;
  const int cap = kept_entries(capacity, N, k, E);
  if (cap < 0) return TOPMOE_ERR_BAD_ARG;
  if (need > 0 && workspace_bytes < need) return TOPMOE_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(x, 16) || !aligned(xs, 16) || !aligned(topk_idx, 4) || !aligned(expert_offsets, 4) ||
      !aligned(row_entry, 4) || !aligned(entry_row, 4) || !aligned(workspace, 256))
    return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch rows = st.at(0), copy = st.at(1);
  TOPMOE_TRY(launch_dispatch_rows(x, topk_idx, N, int(H), E, k, cap, dtype, xs, expert_offsets,
                                  row_entry, entry_row, static_cast<int32_t*>(workspace), rows,
                                  copy));
  TOPMOE_TRY(st.close(rows));
  TOPMOE_TRY(st.close(copy));
  return TOPMOE_OK;
}

// ---- norms
int pieces(int64_t H, int dtype) { return int(H / (dtype == TOPMOE_DTYPE_FP32 ? 4 : 8)); }

int norm_shape(int64_t N, int64_t H, int64_t gate_rows) {
  if (N < 0 || N > kMaxRows) return TOPMOE_ERR_BAD_SHAPE;
  if (H <= 0 || H % 8 != 0 || H > kNormMaxH) return TOPMOE_ERR_BAD_SHAPE;
  if (gate_rows < 0 || gate_rows > kMaxRows || (gate_rows == 0 && N > 0) ||
      (gate_rows > 0 && N % gate_rows != 0))
    return TOPMOE_ERR_BAD_SHAPE;
  return TOPMOE_OK;
}

// Alignment of a gate and its gradient: rows of pieces, or values one by one.
size_t gate_align(int gate_mode, int dtype) {
  if (gate_mode == kGateChannel) return 16;
  return dtype == TOPMOE_DTYPE_FP32 ? 4 : 2;
}

// Tokens that share a row of the gate (the whole batch for the other modes).
int64_t span_of(int64_t N, int64_t gate_rows) {
  const int64_t s = gate_rows > 0 ? N / gate_rows : N;
  return s > 0 ? s : 1;
}

size_t norm_bwd_bytes(const NormUnits& u, int64_t H) {
  return align_up(size_t(2) * size_t(u.count / u.blocks_of) * size_t(H) * sizeof(float) + 1);
}

// ---- 8-bit activations
int act8_shape(int64_t R, int64_t C) {
  if (R < 0 || R > kMaxRows || C <= 0 || C % 8 != 0 || C > kMaxRows) return TOPMOE_ERR_BAD_SHAPE;
  return TOPMOE_OK;
}
// A kept training forward: the routing (MoE), then g and u in 8 bits and their
// scale bytes, each part 256-byte aligned.
struct Keep8 {
  size_t routing = 0, gq = 0, uq = 0, gs = 0, us = 0, total = 0;
};
Keep8 plan_keep8(size_t routing, int64_t rows, int64_t I) {
  Keep8 k;
  const size_t n = size_t(rows) * size_t(I);
  k.routing = routing;
  k.gq = align_up(routing);
  k.uq = align_up(k.gq + n);
  k.gs = align_up(k.uq + n);
  k.us = align_up(k.gs + n / kAct8Group);
  k.total = align_up(k.us + n / kAct8Group + 1);
  return k;
}

// Stage 0: the workspace's routing and pairs into `kept`.
int keep8(const Keep8& k, const void* saved, size_t off_gu, int64_t rows, int64_t I, int dtype,
          void* kept, void* stream, void* const* stage_events) {
  const char* sv = static_cast<const char*>(saved);
  uint8_t* kp = static_cast<uint8_t*>(kept);
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  Launch first = L, second = L;
  const bool both = k.routing > 0 && rows > 0;
  if (both) first.stop = second.start = nullptr;
  if (k.routing > 0) TOPMOE_TRY(launch_copy(sv, kp, k.routing, first));
  if (rows > 0)
    TOPMOE_TRY(launch_pairs_pack(sv + off_gu, rows, I, dtype, kp + k.gq, kp + k.gs, kp + k.uq,
                                 kp + k.us, second));
  L.launched = first.launched || second.launched;
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

// Stage 0: the routing from `kept` (empty for the dense FFN); stage 1: the pairs
// and h^T.
int restore8(const Keep8& k, const void* kept, size_t off_gu, size_t off_hT,
             const int32_t* offsets, int E, int64_t rows, int64_t I, int64_t ldk, int dtype,
             void* workspace, void* stream, void* const* stage_events) {
  const uint8_t* kp = static_cast<const uint8_t*>(kept);
  char* ws = static_cast<char*>(workspace);
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch l0 = st.at(0);
  if (k.routing > 0) TOPMOE_TRY(launch_copy(kp, ws, k.routing, l0));
  TOPMOE_TRY(st.close(l0));
  const Launch l1 = st.at(1);
  const Restore8Job job{kp + k.gq, kp + k.gs, kp + k.uq, kp + k.us, ws + off_gu, ws + off_hT,
                        offsets, E, int(I), rows, ldk};
  TOPMOE_TRY(launch_restore8(dtype, job, l1));
  TOPMOE_TRY(st.close(l1));
  return TOPMOE_OK;
}

// What keep8 / restore8 check of their two buffers.
int keep8_buffers(const void* ws, size_t ws_bytes, size_t ws_need, const void* kept,
                  size_t kept_bytes, size_t kept_need) {
  if (!ws || !kept) return TOPMOE_ERR_NULL_ARG;
  if (ws_bytes < ws_need || kept_bytes < kept_need) return TOPMOE_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 256) || !aligned(kept, 256)) return TOPMOE_ERR_BAD_ARG;
  return TOPMOE_OK;
}

bool pitch_ok(int64_t ld, int64_t C) { return ld >= C && ld % 8 == 0; }

}  // namespace

extern "C" {

size_t moe_dispatch_workspace_bytes(int64_t N, int E, int k) {
  if (E < 1 || E > kDispatchMaxExperts || k > E || rows_shape(N, 8, k) != TOPMOE_OK) return 0;
  return align_up(plan_dispatch(N * k, E).bytes + 1);
}

int moe_dispatch_fwd(const void* x, const int32_t* topk_idx, int64_t N, int64_t H, int E, int k,
                     float capacity_factor, int dtype, void* xs, int32_t* expert_offsets,
                     int32_t* row_entry, int32_t* entry_row, void* workspace,
                     size_t workspace_bytes, void* stream, void* const* stage_events) {
  return dispatch_fwd(x, topk_idx, N, H, E, k, capacity_factor, dtype, xs, expert_offsets,
                      row_entry, entry_row, workspace, workspace_bytes, stream, stage_events);
}

int moe_dispatch_fwd_capacity(const void* x, const int32_t* topk_idx, int64_t N, int64_t H, int E,
                              int k, int64_t capacity, int dtype, void* xs,
                              int32_t* expert_offsets, int32_t* row_entry, int32_t* entry_row,
                              void* workspace, size_t workspace_bytes, void* stream,
                              void* const* stage_events) {
  return dispatch_fwd(x, topk_idx, N, H, E, k, capacity, dtype, xs, expert_offsets, row_entry,
                      entry_row, workspace, workspace_bytes, stream, stage_events);
}

int moe_dispatch_bwd(const void* dxs, const int32_t* entry_row, int64_t N, int64_t H, int k,
                     int dtype, void* dx, void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = rows_shape(N, H, k);
  if (status != TOPMOE_OK) return status;
  if (N > 0 && (!dxs || !entry_row || !dx)) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(dxs, 16) || !aligned(dx, 16) || !aligned(entry_row, 4)) return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_gather_sum(dxs, entry_row, nullptr, nullptr, N, int(H), k, dtype, dx, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

int moe_combine_fwd(const void* ys, const int32_t* entry_row, const float* alpha,
                    const void* residual, int64_t N, int64_t H, int k, int dtype, void* y,
                    void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = rows_shape(N, H, k);
  if (status != TOPMOE_OK) return status;
  if (N > 0 && (!ys || !entry_row || !alpha || !y)) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(ys, 16) || !aligned(residual, 16) || !aligned(y, 16) || !aligned(entry_row, 4) ||
      !aligned(alpha, 4))
    return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_gather_sum(ys, entry_row, alpha, residual, N, int(H), k, dtype, y, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

int moe_combine_bwd(const void* dy, const void* ys, const int32_t* entry_row, const float* alpha,
                    int64_t N, int64_t H, int k, int dtype, void* dys, float* dalpha,
                    void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = rows_shape(N, H, k);
  if (status != TOPMOE_OK) return status;
  if (N > 0 && (!dy || !ys || !entry_row || !alpha || !dys || !dalpha)) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(dy, 16) || !aligned(ys, 16) || !aligned(dys, 16) || !aligned(entry_row, 4) ||
      !aligned(alpha, 4) || !aligned(dalpha, 4))
    return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_moe_combine_bwd(dy, ys, entry_row, alpha, N, int(H), k, dtype, dys, dalpha, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

int block_prenorm_fwd(const void* x, const void* w, int64_t N, int64_t H, float eps, int dtype,
                      void* n, float* rstd, void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = norm_shape(N, H, N > 0 ? 1 : 0);
  if (status != TOPMOE_OK) return status;
  if (!w || (N > 0 && (!x || !n || !rstd))) return TOPMOE_ERR_NULL_ARG;
  if (!(eps > 0.f) || isinf(eps)) return TOPMOE_ERR_BAD_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(n, 16) || !aligned(rstd, 4))
    return TOPMOE_ERR_BAD_ARG;
  NormFwd a{};
  a.y = x; a.next_w = w; a.n = n; a.next_rstd = rstd;
  a.N = N; a.H = int(H); a.hv = pieces(H, dtype); a.eps = eps; a.gate_span = 1;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_norm_fwd(a, false, true, dtype, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

size_t block_norm_bwd_workspace_bytes(int64_t N, int64_t H, int64_t gate_rows) {
  if (norm_shape(N, H, gate_rows) != TOPMOE_OK) return 0;
  size_t most = 0;  // of the two types
  for (int dtype : {TOPMOE_DTYPE_FP32, TOPMOE_DTYPE_BF16}) {
    const NormUnits u = plan_norm_units(N, pieces(H, dtype), gate_rows, span_of(N, gate_rows));
    const size_t b = norm_bwd_bytes(u, H);
    most = b > most ? b : most;
  }
  return most;
}

int block_prenorm_bwd(const void* dn, const void* x, const void* w, const float* rstd,
                      const void* dresidual, int64_t N, int64_t H, int dtype, void* dx, void* dw,
                      void* workspace, size_t workspace_bytes, void* stream,
                      void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = norm_shape(N, H, 1);
  if (status != TOPMOE_OK) return status;
  if (!w || !dw || !workspace || (N > 0 && (!dn || !x || !rstd || !dx))) return TOPMOE_ERR_NULL_ARG;
  NormBwd a{};
  a.gate_span = span_of(N, 1);
  a.units = plan_norm_units(N, pieces(H, dtype), 1, a.gate_span);
  if (workspace_bytes < norm_bwd_bytes(a.units, H)) return TOPMOE_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(dn, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(rstd, 4) ||
      !aligned(dresidual, 16) || !aligned(dx, 16) || !aligned(dw, 16) || !aligned(workspace, 256))
    return TOPMOE_ERR_BAD_ARG;
  a.dout = dresidual; a.dn = dn; a.out = x; a.next_w = w; a.next_rstd = rstd;
  a.dy = dx; a.dnext_w = dw; a.part_next = static_cast<float*>(workspace);
  a.N = N; a.gate_rows = 1; a.H = int(H); a.hv = pieces(H, dtype);
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch rows = st.at(0), sums = st.at(1);
  TOPMOE_TRY(launch_norm_bwd(a, false, true, dtype, rows, sums));
  TOPMOE_TRY(st.close(rows));
  TOPMOE_TRY(st.close(sums));
  return TOPMOE_OK;
}

int block_postnorm_fwd(const void* y, const void* residual, const void* w, const void* gate,
                       const void* next_w, int64_t N, int64_t H, int gate_mode,
                       int64_t gate_rows, float residual_scale, float eps, int dtype, void* out,
                       float* rstd, void* n, float* next_rstd, void* stream,
                       void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  if (gate_mode != kGateNone && gate_mode != kGateChannel && gate_mode != kGateToken)
    return TOPMOE_ERR_BAD_ARG;
  const int status = norm_shape(N, H, gate_mode == kGateChannel ? gate_rows : 1);
  if (status != TOPMOE_OK) return status;
  if (N > 0 && (!y || !residual || !out || (gate_mode != kGateNone && !gate) || (w && !rstd) ||
                (next_w && (!n || !next_rstd))))
    return TOPMOE_ERR_NULL_ARG;
  if (!(eps > 0.f) || isinf(eps) || !isfinite(residual_scale)) return TOPMOE_ERR_BAD_ARG;
  if (!aligned(y, 16) || !aligned(residual, 16) || !aligned(w, 16) ||
      !aligned(gate, gate_align(gate_mode, dtype)) || !aligned(next_w, 16) ||
      !aligned(out, 16) || !aligned(rstd, 4) || !aligned(n, 16) || !aligned(next_rstd, 4))
    return TOPMOE_ERR_BAD_ARG;
  NormFwd a{};
  a.y = y; a.residual = residual; a.w = w; a.gate = gate; a.next_w = next_w;
  a.out = out; a.n = n; a.rstd = rstd; a.next_rstd = next_rstd;
  a.N = N; a.H = int(H); a.hv = pieces(H, dtype); a.gate_mode = gate_mode;
  a.gate_span = span_of(N, gate_mode == kGateChannel ? gate_rows : 1);
  a.scale = residual_scale; a.eps = eps;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_norm_fwd(a, true, next_w != nullptr, dtype, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

int block_postnorm_bwd(const void* dout, const void* dn, const void* y, const void* out,
                       const void* w, const void* gate, const void* next_w, const float* rstd,
                       const float* next_rstd, int64_t N, int64_t H, int gate_mode,
                       int64_t gate_rows, float residual_scale, int dtype, void* dy,
                       void* dresidual, void* dw, void* dgate, void* dnext_w, void* workspace,
                       size_t workspace_bytes, void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  if (gate_mode != kGateNone && gate_mode != kGateChannel && gate_mode != kGateToken)
    return TOPMOE_ERR_BAD_ARG;
  const bool channel = gate_mode == kGateChannel;
  const int status = norm_shape(N, H, channel ? gate_rows : 1);
  if (status != TOPMOE_OK) return status;
  if (!workspace || (w && !dw) || (next_w && !dnext_w) ||
      (channel && gate_rows > 0 && (!gate || !dgate)))
    return TOPMOE_ERR_NULL_ARG;
  if (N > 0 && (!y || !dy || !dresidual || (!dout && !next_w) || (w && !rstd) ||
                (next_w && (!dn || !out || !next_rstd)) ||
                (gate_mode == kGateToken && (!gate || !dgate))))
    return TOPMOE_ERR_NULL_ARG;
  if (!isfinite(residual_scale)) return TOPMOE_ERR_BAD_ARG;
  NormBwd a{};
  a.gate_rows = channel ? gate_rows : 1;
  a.gate_span = span_of(N, a.gate_rows);
  a.units = plan_norm_units(N, pieces(H, dtype), a.gate_rows, a.gate_span);
  if (workspace_bytes < norm_bwd_bytes(a.units, H)) return TOPMOE_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(dout, 16) || !aligned(dn, 16) || !aligned(y, 16) || !aligned(out, 16) ||
      !aligned(w, 16) || !aligned(gate, gate_align(gate_mode, dtype)) || !aligned(next_w, 16) ||
      !aligned(rstd, 4) || !aligned(next_rstd, 4) || !aligned(dy, 16) || !aligned(dresidual, 16) ||
      !aligned(dw, 16) || !aligned(dgate, gate_align(gate_mode, dtype)) || !aligned(dnext_w, 16) ||
      !aligned(workspace, 256))
    return TOPMOE_ERR_BAD_ARG;
  a.dout = dout; a.dn = dn; a.y = y; a.out = out; a.w = w; a.gate = gate; a.next_w = next_w;
  a.rstd = w ? rstd : nullptr; a.next_rstd = next_rstd;
  a.dy = dy; a.dresidual = dresidual; a.dw = w ? dw : nullptr; a.dgate = dgate; a.dnext_w = dnext_w;
  float* part = static_cast<float*>(workspace);
  a.part = w || channel ? part : nullptr;
  a.part_next = part + size_t(a.units.count / a.units.blocks_of) * size_t(H);
  a.N = N; a.H = int(H); a.hv = pieces(H, dtype); a.gate_mode = gate_mode; a.scale = residual_scale;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch rows = st.at(0), sums = st.at(1);
  TOPMOE_TRY(launch_norm_bwd(a, true, next_w != nullptr, dtype, rows, sums));
  TOPMOE_TRY(st.close(rows));
  TOPMOE_TRY(st.close(sums));
  return TOPMOE_OK;
}

int act8_pack(const void* x, int64_t ldx, int64_t R, int64_t C, int dtype, uint8_t* q,
              uint8_t* scale, void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = act8_shape(R, C);
  if (status != TOPMOE_OK) return status;
  if (!pitch_ok(ldx, C)) return TOPMOE_ERR_BAD_SHAPE;
  if (R > 0 && (!x || !q || !scale)) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(x, 16) || !aligned(q, 8)) return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_act8_pack(x, ldx, R, C, dtype, q, scale, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

int act8_unpack(const uint8_t* q, const uint8_t* scale, int64_t R, int64_t C, int dtype, void* x,
                int64_t ldx, void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = act8_shape(R, C);
  if (status != TOPMOE_OK) return status;
  if (!pitch_ok(ldx, C)) return TOPMOE_ERR_BAD_SHAPE;
  if (R > 0 && (!x || !q || !scale)) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(x, 16) || !aligned(q, 8)) return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_act8_unpack(q, scale, R, C, dtype, x, ldx, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

int swiglu_act8_fwd(const void* g, int64_t ldg, const void* u, int64_t ldu, int64_t R, int64_t C,
                    int dtype, void* h, uint8_t* gq, uint8_t* gscale, uint8_t* uq,
                    uint8_t* uscale, void* stream, void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = act8_shape(R, C);
  if (status != TOPMOE_OK) return status;
  if (!pitch_ok(ldg, C) || !pitch_ok(ldu, C)) return TOPMOE_ERR_BAD_SHAPE;
  if (R > 0 && (!g || !u || !h || !gq || !gscale || !uq || !uscale)) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(g, 16) || !aligned(u, 16) || !aligned(h, 16) || !aligned(gq, 8) || !aligned(uq, 8))
    return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_swiglu_act8_fwd(g, ldg, u, ldu, R, C, dtype, h, gq, gscale, uq, uscale, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

int swiglu_act8_bwd(const uint8_t* gq, const uint8_t* gscale, const uint8_t* uq,
                    const uint8_t* uscale, const void* dh, int64_t R, int64_t C, int dtype,
                    void* dg, int64_t lddg, void* du, int64_t lddu, void* h, void* stream,
                    void* const* stage_events) {
  if (!known_dtype(dtype)) return TOPMOE_ERR_UNSUPPORTED_DTYPE;
  const int status = act8_shape(R, C);
  if (status != TOPMOE_OK) return status;
  if (!pitch_ok(lddg, C) || !pitch_ok(lddu, C)) return TOPMOE_ERR_BAD_SHAPE;
  if (R > 0 && (!gq || !gscale || !uq || !uscale || !dh || !dg || !du)) return TOPMOE_ERR_NULL_ARG;
  if (!aligned(gq, 8) || !aligned(uq, 8) || !aligned(dh, 16) || !aligned(dg, 16) ||
      !aligned(du, 16) || !aligned(h, 16))
    return TOPMOE_ERR_BAD_ARG;
  const Stages st{stage_events, static_cast<hipStream_t>(stream)};
  const Launch L = st.at(0);
  TOPMOE_TRY(launch_swiglu_act8_bwd(gq, gscale, uq, uscale, dh, R, C, dtype, dg, lddg, du, lddu,
                                    h, L));
  TOPMOE_TRY(st.close(L));
  return TOPMOE_OK;
}

size_t ffn_keep8_bytes(int64_t N, int64_t H, int64_t I, int dtype) {
  FfnBwdPlan pl;
  return plan_ffn_bwd(N, H, I, dtype, &pl) == TOPMOE_OK ? plan_keep8(0, N, I).total : 0;
}

int ffn_swiglu_keep8(const void* saved, size_t saved_bytes, int64_t N, int64_t H, int64_t I,
                     int dtype, void* kept, size_t kept_bytes, void* stream,
                     void* const* stage_events) {
  FfnBwdPlan pl;
  const int status = plan_ffn_bwd(N, H, I, dtype, &pl);
  if (status != TOPMOE_OK) return status;
  const Keep8 k = plan_keep8(0, N, I);
  const int st = keep8_buffers(saved, saved_bytes, pl.total, kept, kept_bytes, k.total);
  if (st != TOPMOE_OK) return st;
  return keep8(k, saved, pl.off_gu, N, I, dtype, kept, stream, stage_events);
}

int ffn_swiglu_restore8(const void* kept, size_t kept_bytes, int64_t N, int64_t H, int64_t I,
                        int dtype, void* workspace, size_t workspace_bytes, void* stream,
                        void* const* stage_events) {
  FfnBwdPlan pl;
  const int status = plan_ffn_bwd(N, H, I, dtype, &pl);
  if (status != TOPMOE_OK) return status;
  const Keep8 k = plan_keep8(0, N, I);
  const int st = keep8_buffers(workspace, workspace_bytes, pl.total, kept, kept_bytes, k.total);
  if (st != TOPMOE_OK) return st;
  return restore8(k, kept, pl.off_gu, pl.off_hT, nullptr, 1, N, I, pl.ldk, dtype, workspace,
                  stream, stage_events);
}

size_t moe_keep8_bytes(int64_t N, int64_t H, int64_t I, int E, int k, int dtype) {
  MoeBwdPlan pl;
  if (plan_moe_bwd(N, H, I, E, k, dtype, &pl) != TOPMOE_OK) return 0;
  return plan_keep8(pl.off_wgT, pl.route.rows, I).total;
}

int moe_ffn_keep8(const void* saved, size_t saved_bytes, int64_t N, int64_t H, int64_t I, int E,
                  int k, int dtype, void* kept, size_t kept_bytes, void* stream,
                  void* const* stage_events) {
  MoeBwdPlan pl;
  const int status = plan_moe_bwd(N, H, I, E, k, dtype, &pl);
  if (status != TOPMOE_OK) return status;
  const Keep8 kp = plan_keep8(pl.off_wgT, pl.route.rows, I);
  const int st = keep8_buffers(saved, saved_bytes, pl.total, kept, kept_bytes, kp.total);
  if (st != TOPMOE_OK) return st;
  return keep8(kp, saved, pl.off_gu, pl.route.rows, I, dtype, kept, stream, stage_events);
}

int moe_ffn_restore8(const void* kept, size_t kept_bytes, int64_t N, int64_t H, int64_t I, int E,
                     int k, int dtype, void* workspace, size_t workspace_bytes, void* stream,
                     void* const* stage_events) {
  MoeBwdPlan pl;
  const int status = plan_moe_bwd(N, H, I, E, k, dtype, &pl);
  if (status != TOPMOE_OK) return status;
  const Keep8 kp = plan_keep8(pl.off_wgT, pl.route.rows, I);
  const int st = keep8_buffers(workspace, workspace_bytes, pl.total, kept, kept_bytes, kp.total);
  if (st != TOPMOE_OK) return st;
  const int32_t* offsets = reinterpret_cast<const int32_t*>(static_cast<char*>(workspace) +
                                                            pl.route.off_offsets);
  return restore8(kp, kept, pl.off_gu, pl.off_hT, offsets, E, pl.route.rows, I, pl.ldk, dtype,
                  workspace, stream, stage_events);
}

}  // extern "C"
