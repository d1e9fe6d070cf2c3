// C ABI of the block around the adapted layer: the residual RMS norm and the
// matrix product with its epilogue, and their backward passes. Argument
// checks run on the host before anything is enqueued.
#include <math.h>

#include "../../include/dora.h"
#include "dora_check.h"
#include "dora_launch.h"
#include "dora_matmul.h"

using dora::aligned;
using dora::esize;
using dora::hip_status;
using dora::kAlign;
using dora::kMaxDim;
using dora::overlap;
using dora::valid_dtype;

namespace {

// One buffer of a call: its bytes, and the alignment its elements need.
struct Span {
  const void* p;
  int64_t bytes;
  size_t align;
};

// Every element of a tensor is reached with 64-bit arithmetic far from its
// limits, and every launch stays within its grid.
constexpr int64_t kMaxElems = (int64_t)1 << 33;
// Bytes of one row of a product's operand (the tile kernel's 32-bit offsets
// span 256 rows).
constexpr int64_t kMaxRowBytes = (int64_t)1 << 23;
// Rows of a product: 64 of them a workgroup of 256 threads, and a launch takes
// less than 2^32 threads.
constexpr int64_t kMaxRows = (int64_t)1 << 30;

bool size_ok(int64_t a, int64_t b) {
  return a >= 0 && b >= 0 && a < kMaxDim && b < kMaxDim && (b == 0 || a <= kMaxElems / b);
}

// Inputs and outputs are aligned; no output overlaps an input or another
// output, except input i that output o may be exactly (bit i of same[o]).
bool buffers_ok(const Span* in, int n_in, const Span* out, int n_out, const unsigned* same) {
  for (int i = 0; i < n_in; ++i)
    if (!aligned(in[i].p, in[i].align)) return false;
  for (int o = 0; o < n_out; ++o) {
    if (!aligned(out[o].p, out[o].align)) return false;
    for (int i = 0; i < n_in; ++i) {
      if ((same[o] >> i & 1u) && out[o].p == in[i].p) continue;
      if (overlap(out[o].p, out[o].bytes, in[i].p, in[i].bytes)) return false;
    }
    for (int q = o + 1; q < n_out; ++q)
      if (overlap(out[o].p, out[o].bytes, out[q].p, out[q].bytes)) return false;
  }
  return true;
}

dora_status workspace_ok(const void* ws, size_t have, size_t need, const Span* in, int n_in, const Span* out,
                         int n_out) {
  if (need == 0) return DORA_OK;
  if (have < need || ws == nullptr || !aligned(ws, kAlign)) return DORA_ERR_WORKSPACE;
  for (int i = 0; i < n_in; ++i)
    if (overlap(ws, (int64_t)need, in[i].p, in[i].bytes)) return DORA_ERR_INVALID_ARG;
  for (int o = 0; o < n_out; ++o)
    if (overlap(ws, (int64_t)need, out[o].p, out[o].bytes)) return DORA_ERR_INVALID_ARG;
  return DORA_OK;
}

bool valid_act(int act) { return act >= DORA_ACT_NONE && act <= DORA_ACT_SILU; }
int64_t operand_size(int dt) { return dt == DORA_E4M3 ? 1 : esize(dt); }

bool matmul_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t r, int64_t es) {
  return size_ok(M, K) && size_ok(N, K) && size_ok(M, N) && size_ok(M, r) && size_ok(N, r) &&
         M < kMaxRows && K * es < kMaxRowBytes && r * es < kMaxRowBytes && N < kMaxRowBytes;
}

// The backward's products run along M and N too.
bool backward_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t es) {
  return matmul_sizes_ok(M, N, K, 0, es) && M * es < kMaxRowBytes && N * es < kMaxRowBytes;
}

}  // namespace

extern "C" {

dora_status dora_rms_norm(const void* x, const void* residual, const float* weight, float eps, int dtype, int64_t T,
                          int64_t d, void* h, void* y, void* q, float* scale, float* rstd, void* stream) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (!size_ok(T, d) || !isfinite(eps) || !(eps > 0.0f)) return DORA_ERR_INVALID_ARG;
  if (T == 0) return DORA_OK;   // (empty arrays may be null)
  if ((y == nullptr && q == nullptr) || (q == nullptr) != (scale == nullptr)) return DORA_ERR_INVALID_ARG;
  if (residual == nullptr && h != nullptr) return DORA_ERR_INVALID_ARG;
  if (d == 0) return scale == nullptr && rstd == nullptr ? DORA_OK : DORA_ERR_INVALID_ARG;
  if (x == nullptr) return DORA_ERR_INVALID_ARG;
  const int64_t es = esize(dtype), n = T * d;
  const Span in[] = {{x, n * es, (size_t)es}, {residual, n * es, (size_t)es}, {weight, d * 4, 4}};
  const Span out[] = {{h, n * es, (size_t)es}, {y, n * es, (size_t)es}, {q, n, 1}, {scale, T * 4, 4}, {rstd, T * 4, 4}};
  const unsigned same[] = {3u, 0u, 0u, 0u, 0u};   // h may be x or residual itself
  if (!buffers_ok(in, 3, out, 5, same)) return DORA_ERR_INVALID_ARG;
  return hip_status(dora::launch_rms_norm(x, residual, weight, eps, dtype, T, d, h, y, q, scale, rstd,
                                          static_cast<hipStream_t>(stream)));
}

dora_status dora_rms_norm_backward_workspace_size(int64_t T, int64_t d, int dtype, size_t* ws_bytes) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (ws_bytes == nullptr || !size_ok(T, d)) return DORA_ERR_INVALID_ARG;
  *ws_bytes = dora::rms_norm_bwd_workspace_bytes(T, d, dtype);
  return DORA_OK;
}

dora_status dora_rms_norm_backward(const void* dy, const void* dh, const void* h, const float* rstd,
                                   const float* weight, int dtype, int64_t T, int64_t d, void* dx, float* dweight,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (!size_ok(T, d)) return DORA_ERR_INVALID_ARG;
  if (d == 0) return DORA_OK;
  if (T > 0 && (dy == nullptr || h == nullptr || rstd == nullptr || dx == nullptr)) return DORA_ERR_INVALID_ARG;
  const int64_t es = esize(dtype), n = T * d;
  const Span in[] = {{dy, n * es, (size_t)es}, {dh, n * es, (size_t)es}, {h, n * es, (size_t)es}, {rstd, T * 4, 4},
                     {weight, d * 4, 4}};
  const Span out[] = {{dx, n * es, (size_t)es}, {dweight, d * 4, 4}};
  const unsigned same[] = {3u, 0u};   // dx may be dy or dh itself
  if (!buffers_ok(in, 5, out, 2, same)) return DORA_ERR_INVALID_ARG;
  const size_t need = dweight != nullptr ? dora::rms_norm_bwd_workspace_bytes(T, d, dtype) : 0;
  const dora_status st = workspace_ok(workspace, workspace_bytes, need, in, 5, out, 2);
  if (st != DORA_OK) return st;
  return hip_status(dora::launch_rms_norm_bwd(dy, dh, h, rstd, weight, dtype, T, d, dx, dweight, workspace,
                                              static_cast<hipStream_t>(stream)));
}

dora_status dora_matmul_workspace_size(int64_t M, int64_t N, int64_t K, int64_t r, int dtype, int aligned_operands,
                                       size_t* ws_bytes) {
  if (!valid_dtype(dtype) && dtype != DORA_E4M3) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (ws_bytes == nullptr || !matmul_sizes_ok(M, N, K, r, operand_size(dtype))) return DORA_ERR_INVALID_ARG;
  *ws_bytes = M > 0 && N > 0 ? dora::plan_matmul(M, N, K, r, dtype, aligned_operands).ws_bytes : 0;
  return DORA_OK;
}

dora_status dora_matmul_plan_info(int64_t M, int64_t N, int64_t K, int64_t r, int dtype, int aligned_operands,
                                  int64_t* info, int n_info) {
  if (!valid_dtype(dtype) && dtype != DORA_E4M3) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (info == nullptr || n_info < 0 || !matmul_sizes_ok(M, N, K, r, operand_size(dtype))) return DORA_ERR_INVALID_ARG;
  const dora::MatmulPlan p = M > 0 && N > 0 ? dora::plan_matmul(M, N, K, r, dtype, aligned_operands)
                                            : dora::MatmulPlan{};
  const int rows = p.cfg == dora::kTile256 ? 256 : (p.cfg == dora::kTile128 ? 128 : (p.cfg == dora::kTile64 ? 64 : 0));
  const int copies = (p.pack_x ? 1 : 0) | (p.pack_w ? 2 : 0) | (p.pack_t ? 4 : 0) | (p.pack_b ? 8 : 0);
  const int few = p.cfg == dora::kFew8 ? 8 : (p.cfg == dora::kFew16 ? 16 : (p.cfg == dora::kFew32 ? 32 : -1));
  const int64_t vals[] = {M > 0 && N > 0 ? rows : -1, p.splits, copies, (int64_t)p.ws_bytes, few};
  for (int i = 0; i < n_info; ++i) info[i] = i < 5 ? vals[i] : -1;
  return DORA_OK;
}

dora_status dora_matmul(const void* x, const void* w, int dtype, int64_t M, int64_t N, int64_t K,
                        const float* row_scale, const float* col_scale, const void* t, const void* b, int64_t r,
                        float s, const float* bias, int act, const void* residual, int out_dtype, void* y, void* u,
                        void* workspace, size_t workspace_bytes, void* stream) {
  const bool e8 = dtype == DORA_E4M3;
  if (!valid_dtype(dtype) && !e8) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (!valid_dtype(out_dtype) || (!e8 && out_dtype != dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  const int64_t es = operand_size(dtype), os = esize(out_dtype);
  if (!matmul_sizes_ok(M, N, K, r, es) || !valid_act(act) || !isfinite(s)) return DORA_ERR_INVALID_ARG;
  if (e8 && r > 0) return DORA_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return DORA_OK;
  if (y == nullptr || (K > 0 && (x == nullptr || w == nullptr)) || (r > 0 && (t == nullptr || b == nullptr)))
    return DORA_ERR_INVALID_ARG;
  const Span in[] = {{x, M * K * es, (size_t)es}, {w, N * K * es, (size_t)es}, {r > 0 ? t : nullptr, M * r * es, (size_t)es},
                     {r > 0 ? b : nullptr, N * r * es, (size_t)es}, {row_scale, M * 4, 4}, {col_scale, N * 4, 4},
                     {bias, N * 4, 4}, {residual, M * N * os, (size_t)os}};
  const Span out[] = {{y, M * N * os, (size_t)os}, {u, M * N * os, (size_t)os}};
  const unsigned same[] = {1u << 7, 0u};   // y may be residual itself
  if (!buffers_ok(in, 8, out, 2, same)) return DORA_ERR_INVALID_ARG;
  const int al = (aligned(x, 16) ? 1 : 0) | (aligned(w, 16) ? 2 : 0) | (aligned(t, 16) ? 4 : 0) | (aligned(b, 16) ? 8 : 0);
  const dora::MatmulPlan p = dora::plan_matmul(M, N, K, r, dtype, al);
  const dora_status st = workspace_ok(workspace, workspace_bytes, p.ws_bytes, in, 8, out, 2);
  if (st != DORA_OK) return st;
  const dora::Epilogue ep{row_scale, col_scale, bias, residual, y, u, act};
  return hip_status(dora::launch_matmul(p, x, w, dtype, M, N, K, t, b, r, s, ep, out_dtype,
                                        static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
}

dora_status dora_matmul_backward_workspace_size(int64_t M, int64_t N, int64_t K, int dtype, int outputs,
                                                size_t* ws_bytes) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  if (ws_bytes == nullptr || outputs < 0 || outputs >= 2 * DORA_GRAD_ALIGNED ||
      !backward_sizes_ok(M, N, K, esize(dtype)))
    return DORA_ERR_INVALID_ARG;
  *ws_bytes = dora::plan_matmul_backward(M, N, K, dtype, outputs & DORA_GRAD_DX, outputs & DORA_GRAD_DW,
                                         outputs & DORA_GRAD_SUMS, outputs & DORA_GRAD_DU, outputs & DORA_GRAD_ALIGNED)
                  .ws_bytes;
  return DORA_OK;
}

dora_status dora_matmul_backward(const void* dy, const void* u, const void* x, const void* w, int dtype, int64_t M,
                                 int64_t N, int64_t K, const float* col_scale, const float* bias, int act, void* du,
                                 void* dx, void* dw, float* dbias, float* dcol_scale, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  return dora_matmul_backward_rows(dy, u, x, w, dtype, M, N, K, nullptr, col_scale, bias, act, du, dx, dw, dbias,
                                   dcol_scale, workspace, workspace_bytes, stream);
}

dora_status dora_matmul_backward_rows(const void* dy, const void* u, const void* x, const void* w, int dtype,
                                      int64_t M, int64_t N, int64_t K, const float* row_scale, const float* col_scale,
                                      const float* bias, int act, void* du, void* dx, void* dw, float* dbias,
                                      float* dcol_scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype)) return DORA_ERR_UNSUPPORTED_DTYPE;
  const int64_t es = esize(dtype);
  if (!backward_sizes_ok(M, N, K, es) || !valid_act(act)) return DORA_ERR_INVALID_ARG;
  const bool rows = M > 0 && N > 0;
  if (rows && (dy == nullptr || u == nullptr)) return DORA_ERR_INVALID_ARG;
  if (dx != nullptr && N * K > 0 && w == nullptr) return DORA_ERR_INVALID_ARG;
  if (dw != nullptr && M * K > 0 && x == nullptr) return DORA_ERR_INVALID_ARG;
  const size_t e = (size_t)es;
  const Span in[] = {{dy, M * N * es, e}, {u, M * N * es, e}, {dw ? x : nullptr, M * K * es, e},
                     {dx ? w : nullptr, N * K * es, e}, {col_scale, N * 4, 4}, {bias, N * 4, 4}, {row_scale, M * 4, 4}};
  const Span out[] = {{du, M * N * es, e}, {dx, M * K * es, e}, {dw, N * K * es, e}, {dbias, N * 4, 4},
                      {dcol_scale, N * 4, 4}};
  const unsigned same[] = {1u, 0u, 0u, 0u, 0u};   // du may be dy itself
  if (!buffers_ok(in, 7, out, 5, same)) return DORA_ERR_INVALID_ARG;
  const dora::MatmulBackwardPlan p =
      dora::plan_matmul_backward(M, N, K, dtype, dx != nullptr, dw != nullptr, dbias != nullptr || dcol_scale != nullptr,
                                 du != nullptr && aligned(du, 16),
                                 (dw == nullptr || aligned(x, 16)) && (dx == nullptr || aligned(w, 16)));
  const dora_status st = workspace_ok(workspace, workspace_bytes, p.ws_bytes, in, 7, out, 5);
  if (st != DORA_OK) return st;
  return hip_status(dora::launch_matmul_backward(p, dy, u, x, w, dtype, M, N, K, row_scale, col_scale, bias, act, du,
                                                 dx, dw, dbias, dcol_scale, static_cast<char*>(workspace),
                                                 static_cast<hipStream_t>(stream)));
}

}  // extern "C"
