// Kernel launchers behind the C ABI (host side, defined in the .hip files).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dora_plan.h"

namespace dora {

// Timing marks of one norm call: ev[0] is recorded on the stream before the
// call's first launch and ev[i] after its i-th launch, for i < n; null
// entries are skipped. Lives on the caller's stack for one call.
struct Marks {
  const hipEvent_t* ev;
  int n;
  int next;
};
constexpr int kMaxLaunchEvents = 8;

hipError_t launch_norm_factored(const NormPlan& p, const void* W, const void* A, const void* B, void* ws,
                                float s, const float* m, float eps, float* wnorm, float* g, hipStream_t st,
                                const hipEvent_t* events, int n_events);
hipError_t launch_norm_dense(const NormPlan& p, const void* W, const void* A, const void* B, void* ws, float s,
                             const float* m, float eps, float* wnorm, float* g, hipStream_t st,
                             const hipEvent_t* events, int n_events);
hipError_t launch_norm_rowonly(const void* W, int dtype, int64_t d_out, int64_t d_in, bool vec, const float* m,
                               float eps, float* wnorm, float* g, hipStream_t st, const hipEvent_t* events,
                               int n_events);
hipError_t launch_magnitude(const float* m, const float* wnorm, float eps, int64_t n, float* g, hipStream_t st);
hipError_t launch_cast(const float* wnorm, int64_t n, int dtype, void* out, hipStream_t st);
hipError_t launch_compose(const void* base, const void* lora, const float* g, float s, int dtype, int64_t T,
                          int64_t d_out, void* out, bool vec, bool add_base, hipStream_t st);
size_t compose_bwd_workspace_bytes(int64_t T, int64_t d_out);
hipError_t launch_compose_bwd(const void* dy, const void* base, const void* lora, const float* g, float s, int dtype,
                              int64_t T, int64_t d_out, void* d_base, void* d_lora, float* dg, const float* wnorm,
                              float eps, float* dm, void* ws, bool vec, hipStream_t st);
hipError_t launch_column_sum(const float* part, int n_part, int64_t n, float* out0, int64_t n0, float* out1,
                             hipStream_t st);
hipError_t launch_rms_norm(const void* x, const void* residual, const float* weight, float eps, int dtype, int64_t T,
                           int64_t d, void* h, void* y, void* q, float* scale, float* rstd, hipStream_t st);
size_t rms_norm_bwd_workspace_bytes(int64_t T, int64_t d, int dtype);
hipError_t launch_rms_norm_bwd(const void* dy, const void* dh, const void* h, const float* rstd, const float* weight,
                               int dtype, int64_t T, int64_t d, void* dx, float* dweight, void* ws, hipStream_t st);
// Rows in 8-bit integers: q [rows][d] and the scales of each row's groups of
// `group` columns (0: one scale a row).
struct Int8Rows {
  const uint8_t* q;
  const float* scale;
  int64_t group;
};
// Scales of a row, and log2 of a group's columns (62 where the row is one).
inline int64_t scales_of(int64_t d, int64_t group) { return group ? (d + group - 1) / group : 1; }
inline int group_shift(int64_t group) {
  int s = 0;
  while (group && ((int64_t)1 << s) < group) ++s;
  return group ? s : 62;
}
hipError_t launch_layer_norm(const void* x, const void* residual, const float* weight, const float* bias, float eps,
                             int dtype, int64_t T, int64_t d, void* h, void* y, void* q, int q_int8, float* scale,
                             float* mean, float* rstd, hipStream_t st);
size_t layer_norm_bwd_workspace_bytes(int64_t T, int64_t d, int dtype);
hipError_t launch_layer_norm_bwd(const void* dy, const void* dh, const void* h, const float* mean, const float* rstd,
                                 const float* weight, int dtype, int64_t T, int64_t d, void* dx, float* dweight,
                                 float* dbias, void* ws, hipStream_t st);
hipError_t launch_quantize_rows(const void* x, int dtype, int64_t T, int64_t d, int64_t group, void* q, float* scale,
                                hipStream_t st);
hipError_t launch_dequantize_rows(const Int8Rows& r, int64_t T, int64_t d, int dtype, void* x, hipStream_t st);
size_t fast_kernel_lds_bytes(int cfg);
size_t gen_kernel_lds_bytes(int cfg);

}  // namespace dora
