// C ABI of the layer norm and of rows held in 8-bit integers: packing, the
// integer product, and the backward that reads packed operands. Argument
// checks run on the host before anything is enqueued.
#include "../../include/dora.h"
#include "block_check.h"
#include "dora_launch.h"
#include "dora_matmul.h"

using namespace dora;

namespace {

// Longest depth whose sum of products of 8-bit integers cannot pass int32.
constexpr int64_t kMaxInt8Depth = 131071;

bool group_ok(int64_t g) { return g == 0 || g == 32 || g == 64 || g == 128 || g == 256; }

bool int8_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t r) {
  return matmul_sizes_ok(M, N, K, 0, 1) && matmul_sizes_ok(M, N, 0, r, 2) && K <= kMaxInt8Depth;
}

MatmulPlan int8_plan(int64_t M, int64_t N, int64_t K, int64_t r, int al) {
  return plan_matmul(M, N, K, r, kInt8Operands, al);
}

// One operand of the backward, in the storage type or as int8 rows, which are
// two buffers.
bool held_ok(const void* v, const dora_int8_rows* r, bool read, bool empty) {
  if (!read) return true;
  if (r == nullptr) return v != nullptr || empty;
  return v == nullptr && group_ok(r->group) && (empty || (r->q != nullptr && r->scale != nullptr));
}

// An operand's form, by how many scales a row of it has (0: it is not held so).
HeldForm form_of(int64_t scales) { return scales == 0 ? kNotHeld : (scales > 1 ? kHeldGroups : kHeldRows); }
HeldForm form_of(const dora_int8_rows* r, int64_t columns) {
  return r == nullptr ? kNotHeld : (scales_of(columns, r->group) > 1 ? kHeldGroups : kHeldRows);
}

Int8Rows rows_of(const dora_int8_rows* r, bool read) {
  return r != nullptr && read ? Int8Rows{reinterpret_cast<const uint8_t*>(r->q), r->scale, r->group} : Int8Rows{};
}

}  // namespace

extern "C" {

dora_status dora_layer_norm(const void* x, const void* residual, const float* weight, const float* bias, float eps,
                            int dtype, int64_t T, int64_t d, void* h, void* y, void* q, int q_dtype, float* scale,
                            float* mean, float* rstd, void* stream) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (q != nullptr && q_dtype != DORA_E4M3 && q_dtype != DORA_I8) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (!size_ok(T, d) || !isfinite(eps) || !(eps > 0.0f)) return DORA_ERR_INVALID_ARG;
  if (T == 0) return DORA_OK;   // (empty arrays may be null)
  if ((y == nullptr && q == nullptr) || (q == nullptr) != (scale == nullptr)) return DORA_ERR_INVALID_ARG;
  if (residual == nullptr && h != nullptr) return DORA_ERR_INVALID_ARG;
  if (d == 0) return scale == nullptr && mean == nullptr && rstd == nullptr ? DORA_OK : DORA_ERR_INVALID_ARG;
  if (x == nullptr) return DORA_ERR_INVALID_ARG;
  const int64_t es = esize(dtype), n = T * d;
  const Span in[] = {{x, n * es, (size_t)es}, {residual, n * es, (size_t)es}, {weight, d * 4, 4}, {bias, d * 4, 4}};
  const Span out[] = {{h, n * es, (size_t)es}, {y, n * es, (size_t)es}, {q, n, 1}, {scale, T * 4, 4}, {mean, T * 4, 4},
                      {rstd, T * 4, 4}};
  const unsigned same[] = {3u, 0u, 0u, 0u, 0u, 0u};   // h may be x or residual itself
  if (!buffers_ok(in, 4, out, 6, same)) return DORA_ERR_INVALID_ARG;
  return hip_status(launch_layer_norm(x, residual, weight, bias, eps, dtype, T, d, h, y, q, q_dtype == DORA_I8, scale,
                                      mean, rstd, static_cast<hipStream_t>(stream)));
}

dora_status dora_layer_norm_backward_workspace_size(int64_t T, int64_t d, int dtype, size_t* ws_bytes) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (ws_bytes == nullptr || !size_ok(T, d)) return DORA_ERR_INVALID_ARG;
  *ws_bytes = layer_norm_bwd_workspace_bytes(T, d, dtype);
  return DORA_OK;
}

dora_status dora_layer_norm_backward(const void* dy, const void* dh, const void* h, const float* mean,
                                     const float* rstd, const float* weight, int dtype, int64_t T, int64_t d, void* dx,
                                     float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (!size_ok(T, d)) return DORA_ERR_INVALID_ARG;
  if (d == 0) return DORA_OK;
  if (T > 0 && (dy == nullptr || h == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr))
    return DORA_ERR_INVALID_ARG;
  const int64_t es = esize(dtype), n = T * d;
  const Span in[] = {{dy, n * es, (size_t)es}, {dh, n * es, (size_t)es}, {h, n * es, (size_t)es}, {mean, T * 4, 4},
                     {rstd, T * 4, 4}, {weight, d * 4, 4}};
  const Span out[] = {{dx, n * es, (size_t)es}, {dweight, d * 4, 4}, {dbias, d * 4, 4}};
  const unsigned same[] = {3u, 0u, 0u};   // dx may be dy or dh itself
  if (!buffers_ok(in, 6, out, 3, same)) return DORA_ERR_INVALID_ARG;
  const bool sums = dweight != nullptr || dbias != nullptr;
  const size_t need = sums ? layer_norm_bwd_workspace_bytes(T, d, dtype) : 0;
  const dora_status st = workspace_ok(workspace, workspace_bytes, need, in, 6, out, 3);
  if (st != DORA_OK) return st;
  return hip_status(launch_layer_norm_bwd(dy, dh, h, mean, rstd, weight, dtype, T, d, dx, dweight, dbias, workspace,
                                          static_cast<hipStream_t>(stream)));
}

dora_status dora_quantize_rows(const void* x, int dtype, int64_t T, int64_t d, int64_t group, int8_t* q, float* scale,
                               void* stream) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (!size_ok(T, d) || !group_ok(group)) return DORA_ERR_INVALID_ARG;
  if (T == 0) return DORA_OK;
  if (d == 0) return group == 0 ? DORA_ERR_INVALID_ARG : DORA_OK;
  if (x == nullptr || q == nullptr || scale == nullptr) return DORA_ERR_INVALID_ARG;
  const int64_t es = esize(dtype);
  const Span in[] = {{x, T * d * es, (size_t)es}};
  const Span out[] = {{q, T * d, 1}, {scale, T * scales_of(d, group) * 4, 4}};
  const unsigned same[] = {0u, 0u};
  if (!buffers_ok(in, 1, out, 2, same)) return DORA_ERR_INVALID_ARG;
  return hip_status(launch_quantize_rows(x, dtype, T, d, group, q, scale, static_cast<hipStream_t>(stream)));
}

dora_status dora_dequantize_rows(const int8_t* q, const float* scale, int64_t T, int64_t d, int64_t group, int dtype,
                                 void* x, void* stream) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (!size_ok(T, d) || !group_ok(group)) return DORA_ERR_INVALID_ARG;
  if (T == 0 || d == 0) return DORA_OK;
  if (x == nullptr || q == nullptr || scale == nullptr) return DORA_ERR_INVALID_ARG;
  const int64_t es = esize(dtype);
  const Span in[] = {{q, T * d, 1}, {scale, T * scales_of(d, group) * 4, 4}};
  const Span out[] = {{x, T * d * es, (size_t)es}};
  const unsigned same[] = {0u};
  if (!buffers_ok(in, 2, out, 1, same)) return DORA_ERR_INVALID_ARG;
  return hip_status(launch_dequantize_rows(Int8Rows{reinterpret_cast<const uint8_t*>(q), scale, group}, T, d, dtype, x,
                                           static_cast<hipStream_t>(stream)));
}

dora_status dora_matmul_int8_workspace_size(int64_t M, int64_t N, int64_t K, int64_t r, int aligned_operands,
                                            size_t* ws_bytes) {
  if (ws_bytes == nullptr || !int8_sizes_ok(M, N, K, r)) return DORA_ERR_INVALID_ARG;
  *ws_bytes = M > 0 && N > 0 ? int8_plan(M, N, K, r, aligned_operands).ws_bytes : 0;
  return DORA_OK;
}

dora_status dora_matmul_int8_plan_info(int64_t M, int64_t N, int64_t K, int64_t r, int aligned_operands, int64_t* info,
                                       int n_info) {
  if (info == nullptr || n_info < 0 || !int8_sizes_ok(M, N, K, r)) return DORA_ERR_INVALID_ARG;
  const bool any = M > 0 && N > 0;
  plan_fields(any ? int8_plan(M, N, K, r, aligned_operands) : MatmulPlan{}, any, true, info, n_info);
  return DORA_OK;
}

dora_status dora_matmul_int8(const int8_t* x, const float* row_scale, const int8_t* w, const float* w_scale, int64_t M,
                             int64_t N, int64_t K, const float* col_scale, const void* t, const void* b, int64_t r,
                             float s, const float* bias, int act, const void* residual, int out_dtype, void* y, void* u,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(out_dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (!int8_sizes_ok(M, N, K, r) || !valid_act(act) || !isfinite(s)) return DORA_ERR_INVALID_ARG;
  if (r > 0 && out_dtype == DORA_F32) return DORA_ERR_INVALID_ARG;
  if (r > 0 && s != 0.f && (fabsf(s) < 0x1p-64f || fabsf(s) > 0x1p64f)) return DORA_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return DORA_OK;
  if (y == nullptr || row_scale == nullptr || w_scale == nullptr || (K > 0 && (x == nullptr || w == nullptr)) ||
      (r > 0 && (t == nullptr || b == nullptr)))
    return DORA_ERR_INVALID_ARG;
  const int64_t os = esize(out_dtype);
  const Span in[] = {{x, M * K, 1}, {w, N * K, 1}, {r > 0 ? t : nullptr, M * r * 2, 2}, {r > 0 ? b : nullptr, N * r * 2, 2},
                     {row_scale, M * 4, 4}, {w_scale, N * 4, 4}, {col_scale, N * 4, 4}, {bias, N * 4, 4},
                     {residual, M * N * os, (size_t)os}};
  const Span out[] = {{y, M * N * os, (size_t)os}, {u, M * N * os, (size_t)os}};
  const unsigned same[] = {1u << 8, 0u};   // y may be residual itself
  if (!buffers_ok(in, 9, out, 2, same)) return DORA_ERR_INVALID_ARG;
  const int al = (aligned(x, 16) ? 1 : 0) | (aligned(w, 16) ? 2 : 0) | (aligned(t, 16) ? 4 : 0) | (aligned(b, 16) ? 8 : 0);
  const int64_t pair = s == 0.f ? 0 : r;
  const MatmulPlan p = int8_plan(M, N, K, pair, al);
  const dora_status st = workspace_ok(workspace, workspace_bytes, p.ws_bytes, in, 9, out, 2);
  if (st != DORA_OK) return st;
  const Epilogue ep{row_scale, col_scale, bias, residual, y, u, act};
  return hip_status(launch_matmul(p, x, w, kInt8Operands, M, N, K, t, b, pair, s, ep, w_scale, out_dtype,
                                  static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
}

dora_status dora_matmul_backward_int8_workspace_size(int64_t M, int64_t N, int64_t K, int dtype, int outputs, int held,
                                                     size_t* ws_bytes) {
  if (held < 0 || held >= 2 * DORA_HELD_W) return DORA_ERR_INVALID_ARG;
  return dora_matmul_backward_int8_scales_workspace_size(M, N, K, dtype, outputs, held & DORA_HELD_X ? 1 : 0,
                                                         held & DORA_HELD_W ? 1 : 0, ws_bytes);
}

dora_status dora_matmul_backward_int8_scales_workspace_size(int64_t M, int64_t N, int64_t K, int dtype, int outputs,
                                                            int64_t x_scales, int64_t w_scales, size_t* ws_bytes) {
  if (ws_bytes == nullptr) return DORA_ERR_INVALID_ARG;
  int64_t info[7];
  const dora_status st = dora_matmul_backward_int8_plan_info(M, N, K, dtype, outputs, x_scales, w_scales, info, 7);
  if (st == DORA_OK) *ws_bytes = (size_t)info[6];
  return st;
}

dora_status dora_matmul_backward_int8_plan_info(int64_t M, int64_t N, int64_t K, int dtype, int outputs,
                                                int64_t x_scales, int64_t w_scales, int64_t* info, int n_info) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (info == nullptr || n_info < 0 || outputs < 0 || outputs >= 2 * DORA_GRAD_ALIGNED || x_scales < 0 ||
      w_scales < 0 || !backward_sizes_ok(M, N, K, esize(dtype)))
    return DORA_ERR_INVALID_ARG;
  const MatmulBackwardPlan p = plan_matmul_backward(
      M, N, K, dtype, outputs & DORA_GRAD_DX, outputs & DORA_GRAD_DW, outputs & DORA_GRAD_SUMS, outputs & DORA_GRAD_DU,
      outputs & DORA_GRAD_ALIGNED, form_of(x_scales), form_of(w_scales));
  const bool dx = (outputs & DORA_GRAD_DX) && M > 0 && K > 0, dw = (outputs & DORA_GRAD_DW) && N > 0 && K > 0;
  const int w = p.w8_tile ? 2 : (p.w8 || p.copy || !p.direct ? 1 : 0), x = p.x8_tile ? 2 : (p.x8 || p.copy || !p.direct ? 1 : 0);
  const int64_t vals[] = {dx ? plan_tile_rows(p.cfg_dx) : -1, dx ? p.splits_dx : -1, dx ? w : -1,
                          dw ? plan_tile_rows(p.cfg_dw) : -1, dw ? p.splits_dw : -1, dw ? x : -1, (int64_t)p.ws_bytes};
  for (int i = 0; i < n_info; ++i) info[i] = i < 7 ? vals[i] : -1;
  return DORA_OK;
}

dora_status dora_matmul_backward_int8(const void* dy, const void* u, const dora_int8_rows* u8, const void* x,
                                      const dora_int8_rows* x8, const void* w, const dora_int8_rows* w8, int dtype,
                                      int64_t M, int64_t N, int64_t K, const float* row_scale, const float* col_scale,
                                      const float* bias, int act, void* du, void* dx, void* dw, float* dbias,
                                      float* dcol_scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  const int64_t es = esize(dtype);
  if (!backward_sizes_ok(M, N, K, es) || !valid_act(act)) return DORA_ERR_INVALID_ARG;
  const bool rows = M > 0 && N > 0;
  if (rows && dy == nullptr) return DORA_ERR_INVALID_ARG;
  if (!held_ok(u, u8, true, !rows) || !held_ok(x, x8, dw != nullptr, M * K == 0) ||
      !held_ok(w, w8, dx != nullptr, N * K == 0))
    return DORA_ERR_INVALID_ARG;
  const HeldInt8 held{rows_of(u8, true), rows_of(x8, dw != nullptr), rows_of(w8, dx != nullptr)};
  const size_t e = (size_t)es;
  const Span in[] = {{dy, M * N * es, e}, {u, M * N * es, e}, {dw ? x : nullptr, M * K * es, e},
                     {dx ? w : nullptr, N * K * es, e}, {col_scale, N * 4, 4}, {bias, N * 4, 4}, {row_scale, M * 4, 4},
                     {held.u.q, M * N, 1}, {held.u.scale, M * scales_of(N, held.u.group) * 4, 4},
                     {held.x.q, M * K, 1}, {held.x.scale, M * scales_of(K, held.x.group) * 4, 4},
                     {held.w.q, N * K, 1}, {held.w.scale, N * scales_of(K, held.w.group) * 4, 4}};
  const Span out[] = {{du, M * N * es, e}, {dx, M * K * es, e}, {dw, N * K * es, e}, {dbias, N * 4, 4},
                      {dcol_scale, N * 4, 4}};
  const unsigned same[] = {1u, 0u, 0u, 0u, 0u};   // du may be dy itself
  if (!buffers_ok(in, 13, out, 5, same)) return DORA_ERR_INVALID_ARG;
  // (of each operand the form that is given; the other one is null)
  const bool al = (dw == nullptr || (aligned(x, 16) && aligned(held.x.q, 16))) &&
                  (dx == nullptr || (aligned(w, 16) && aligned(held.w.q, 16)));
  const MatmulBackwardPlan p =
      plan_matmul_backward(M, N, K, dtype, dx != nullptr, dw != nullptr, dbias != nullptr || dcol_scale != nullptr,
                           du != nullptr && aligned(du, 16), al, form_of(x8, K), form_of(w8, K));
  const dora_status st = workspace_ok(workspace, workspace_bytes, p.ws_bytes, in, 13, out, 5);
  if (st != DORA_OK) return st;
  return hip_status(launch_matmul_backward(p, dy, u, x, w, dtype, M, N, K, row_scale, col_scale, bias, act, du, dx, dw,
                                           dbias, dcol_scale, held, static_cast<char*>(workspace),
                                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"
