// Residual root-mean-square norm on gfx950, with an optional 8-bit output,
// and its backward.
//
//   h = x + residual                 rstd = 1 / sqrt(mean_j h^2 + eps)
//   n[t,j] = h[t,j] rstd[t] w[j]     y = n, rounded once, or
//   scale[t] = max_j |n[t,j]| / 448  q = n / scale in e4m3, rounded once
//
// The norm is of the fp32 sum x + residual; the stored h is that sum rounded
// to the storage type, and nothing is computed from it.
//
// HBM bound: about five operations an element against 5 to 8 bytes. One pass:
// a row is read once into the registers of one wave or one workgroup as
// 16-byte chunks, summed, scaled and written. Rows of any length and
// alignment take the same 16-byte loads and stores (gfx950 reads and writes
// them at any element address); only a row's last partial chunk goes element
// by element. Rows too long for the registers are read again for each step.
// Measured: 8192 x 8192 bf16 to 8 bits 79 us, 5.9 TB/s (to bf16 6.05 TB/s);
// its backward at 8192 x 4096 50 us with the weight's gradient, 5.3 TB/s.
#include "dora_launch.h"
#include "dora_rows.h"

namespace dora {

namespace {

struct NormArgs {
  const void* x;
  const void* residual;
  const float* weight;
  float eps;
  int64_t T, d;
  void* h;
  void* y;
  uint8_t* q;
  float* scale;
  float* rstd;
};

// NT threads and C chunks a thread to a row; workgroups of 256 threads hold
// 256 / NT rows where NT is 64. A workgroup walks rows gridDim.x apart: its
// weights are read once, and a row's loads go out before the row ahead of it
// is reduced.
template <typename T, int NT, int C, bool STREAM, bool LINES>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void rms_norm_kernel(NormArgs a) {
  constexpr int E = Elem<T>::epc;
  // (two sets of words: a wave one row ahead uses the other one)
  __shared__ float red[2][NT > 64 ? 2 * (NT / 64) : 1];
  const int lane = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  constexpr int RPW = NT == 64 ? 4 : 1;   // rows a workgroup holds at a time
  int par = 0;
  const int64_t t0 = (int64_t)blockIdx.x * RPW + (NT == 64 ? threadIdx.x >> 6 : 0);
  const bool has_res = a.residual != nullptr;
  u32x4 xv[C], rv[C];
  auto load = [&](int64_t t) __attribute__((always_inline)) {
    const T* x = static_cast<const T*>(a.x) + t * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c) xv[c] = load_row_chunk<T, STREAM && LINES>(x, (int64_t)(c * NT + lane) * E, a.d);
    if (has_res) {
      const T* res = static_cast<const T*>(a.residual) + t * a.d;
#pragma unroll
      for (int c = 0; c < C; ++c) rv[c] = load_row_chunk<T, STREAM && LINES>(res, (int64_t)(c * NT + lane) * E, a.d);
    }
  };
  if (t0 < a.T) load(t0);
  float w[C][E];
#pragma unroll
  for (int c = 0; c < C; ++c) load_weight<E>(a.weight, (int64_t)(c * NT + lane) * E, a.d, w[c]);
  for (int64_t t = t0; t < a.T; t += (int64_t)gridDim.x * RPW, par ^= 1) {
    float f[C][E], q = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      unpack<T, E>(xv[c], f[c]);
      if (has_res) {
        float r[E];
        unpack<T, E>(rv[c], r);
#pragma unroll
        for (int e = 0; e < E; ++e) f[c][e] += r[e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) q = fmaf(f[c][e], f[c][e], q);
    }
    // (h may be x or residual itself: other rows' loads are of other rows)
    if (t + (int64_t)gridDim.x * RPW < a.T) load(t + (int64_t)gridDim.x * RPW);
    if (a.h) {
      T* h = static_cast<T*>(a.h) + t * a.d;
#pragma unroll
      for (int c = 0; c < C; ++c) store_row_chunk<T, STREAM>(h, (int64_t)(c * NT + lane) * E, a.d, f[c]);
    }
    q = row_sum<NT>(q, red[par]);
    const float rs = 1.f / sqrtf(q / (float)a.d + a.eps);
    if (lane == 0 && a.rstd) a.rstd[t] = rs;
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k = (int64_t)(c * NT + lane) * E;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        f[c][e] = f[c][e] * rs * w[c][e];
        // (past d the row is 0 * rs * w: it counts only where it exists)
        const uint32_t b = k + e < a.d ? abs_bits(f[c][e]) : 0u;
        top = b > top ? b : top;
      }
    }
    if (a.y) {
      T* y = static_cast<T*>(a.y) + t * a.d;
#pragma unroll
      for (int c = 0; c < C; ++c) store_row_chunk<T, STREAM>(y, (int64_t)(c * NT + lane) * E, a.d, f[c]);
    }
    if (a.q) {   // uniform over the grid
      top = row_max_bits<NT>(top, reinterpret_cast<uint32_t*>(red[par]) + (NT > 64 ? NT / 64 : 0));
      const float s = scale_of(top);
      const RowQuotient quotient(s);
      if (lane == 0) a.scale[t] = s;
      uint8_t* qr = a.q + t * a.d;
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int e = 0; e < E; ++e) f[c][e] = quotient(f[c][e]);
        store_row_q<E, STREAM>(qr, (int64_t)(c * NT + lane) * E, a.d, f[c]);
      }
    }
  }
}

// Rows of any length: the row is read once for its sum, once for its largest
// |n| and once to be written (h is written last, so that it may be x or
// residual itself).
template <typename T>
__global__ __launch_bounds__(1024) void rms_norm_long_kernel(NormArgs a) {
  constexpr int E = Elem<T>::epc, NT = 1024;
  __shared__ float red[2][2 * (NT / 64)];
  int par = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
    const T* x = static_cast<const T*>(a.x) + t * a.d;
    const T* res = a.residual ? static_cast<const T*>(a.residual) + t * a.d : nullptr;
    auto load = [&](int64_t k, float (&f)[E]) __attribute__((always_inline)) {
      unpack<T, E>(load_row_chunk(x, k, a.d), f);
      if (res) {
        float r[E];
        unpack<T, E>(load_row_chunk(res, k, a.d), r);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] += r[e];
      }
    };
    float q = 0.f;
    for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
      float f[E];
      load(k, f);
#pragma unroll
      for (int e = 0; e < E; ++e) q = fmaf(f[e], f[e], q);
    }
    q = row_sum<NT>(q, red[par]);
    const float rs = 1.f / sqrtf(q / (float)a.d + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[t] = rs;
    float s = 1.f;
    if (a.q) {
      uint32_t top = 0;
      for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
        float f[E], w[E];
        load(k, f);
        load_weight<E>(a.weight, k, a.d, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t b = k + e < a.d ? abs_bits(f[e] * rs * w[e]) : 0u;
          top = b > top ? b : top;
        }
      }
      top = row_max_bits<NT>(top, reinterpret_cast<uint32_t*>(red[par]) + NT / 64);
      s = scale_of(top);
      if (threadIdx.x == 0) a.scale[t] = s;
    }
    const RowQuotient quotient(s);
    for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
      float f[E], w[E];
      load(k, f);
      if (a.h) store_row_chunk<T>(static_cast<T*>(a.h) + t * a.d, k, a.d, f);
      load_weight<E>(a.weight, k, a.d, w);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = f[e] * rs * w[e];
      if (a.y) store_row_chunk<T>(static_cast<T*>(a.y) + t * a.d, k, a.d, f);
      if (a.q) {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = quotient(f[e]);
        store_row_q<E>(a.q + t * a.d, k, a.d, f);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward. With nh = h rstd and a = dy w:
//   dx[t,j]    = rstd (a - nh mean_j(a nh)) + dh[t,j]
//   dweight[j] = sum_t dy nh
// dx is the gradient of x and of the residual alike. A workgroup walks rows
// blockIdx.x, + gridDim.x, ...; it holds its columns' weights and dweight
// sums in registers (rows in increasing order) and stores one partial row at
// its end; a second kernel adds the partials in a fixed order.
// ---------------------------------------------------------------------------
struct NormBwdArgs {
  const void* dy;
  const void* dh;
  const void* h;
  const float* rstd;
  const float* weight;
  int64_t T, d;
  void* dx;
  float* part;   // [gridDim.x][d], or null
};

template <typename T, int NT, int C, bool STREAM>
__global__ __launch_bounds__(NT) void rms_norm_bwd_kernel(NormBwdArgs a) {
  constexpr int E = Elem<T>::epc;
  __shared__ float red[2][NT > 64 ? NT / 64 : 1];
  const int lane = threadIdx.x;
  float w[C][E], dw[C][E];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_weight<E>(a.weight, (int64_t)(c * NT + lane) * E, a.d, w[c]);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[c][e] = 0.f;
  }
  int par = 0;   // which words the row's sum goes through: a wave a row ahead uses the other ones
  u32x4 yv[2][C], hv[2][C], gv[2][C];
  float rs2[2];
  // (a row's loads go out before the row ahead of it is reduced)
  auto load = [&](int64_t t, u32x4 (&y)[C], u32x4 (&h)[C], u32x4 (&g)[C], float& rs) __attribute__((always_inline)) {
    const T* dyr = static_cast<const T*>(a.dy) + t * a.d;
    const T* hr = static_cast<const T*>(a.h) + t * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      y[c] = load_row_chunk<T, STREAM>(dyr, (int64_t)(c * NT + lane) * E, a.d);
      h[c] = load_row_chunk<T, STREAM>(hr, (int64_t)(c * NT + lane) * E, a.d);
    }
    if (a.dh) {
      const T* gr = static_cast<const T*>(a.dh) + t * a.d;
#pragma unroll
      for (int c = 0; c < C; ++c) g[c] = load_row_chunk<T, STREAM>(gr, (int64_t)(c * NT + lane) * E, a.d);
    }
    rs = a.rstd[t];
  };
  auto row = [&](int64_t t, const u32x4 (&yr)[C], const u32x4 (&hr)[C], const u32x4 (&gr)[C], float rs)
      __attribute__((always_inline)) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float y[E], n[E];
      unpack<T, E>(yr[c], y);
      unpack<T, E>(hr[c], n);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        n[e] *= rs;
        dw[c][e] = fmaf(y[e], n[e], dw[c][e]);
        sum = fmaf(y[e] * w[c][e], n[e], sum);
      }
    }
    const float mean = row_sum<NT>(sum, red[par]) / (float)a.d;
    par ^= 1;
    T* dxr = static_cast<T*>(a.dx) + t * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float y[E], n[E], o[E];
      unpack<T, E>(yr[c], y);
      unpack<T, E>(hr[c], n);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = rs * fmaf(-(n[e] * rs), mean, y[e] * w[c][e]);
      if (a.dh) {
        float g[E];
        unpack<T, E>(gr[c], g);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += g[e];
      }
      store_row_chunk<T>(dxr, (int64_t)(c * NT + lane) * E, a.d, o);
    }
  };
  const int64_t step = gridDim.x;
  int64_t t = blockIdx.x;
  if constexpr (C > 2) {   // (no registers for a second row)
    for (; t < a.T; t += step) {
      load(t, yv[0], hv[0], gv[0], rs2[0]);
      row(t, yv[0], hv[0], gv[0], rs2[0]);
    }
  } else {
    if (t < a.T) load(t, yv[0], hv[0], gv[0], rs2[0]);
    for (; t < a.T; t += 2 * step) {
      if (t + step < a.T) load(t + step, yv[1], hv[1], gv[1], rs2[1]);
      row(t, yv[0], hv[0], gv[0], rs2[0]);
      if (t + step >= a.T) break;
      if (t + 2 * step < a.T) load(t + 2 * step, yv[0], hv[0], gv[0], rs2[0]);
      row(t + step, yv[1], hv[1], gv[1], rs2[1]);
    }
  }
  if (a.part) {
    float* p = a.part + (int64_t)blockIdx.x * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float v[4] = {dw[c][4 * i], dw[c][4 * i + 1], dw[c][4 * i + 2], dw[c][4 * i + 3]};
        store_row_chunk<float>(p, (int64_t)(c * NT + lane) * E + 4 * i, a.d, v);
      }
  }
}

// Rows of any length: each row is read twice, and the workgroup's dweight
// sums live in its partial row in memory (a thread adds to its own columns
// only, rows in increasing order).
template <typename T>
__global__ __launch_bounds__(1024) void rms_norm_bwd_long_kernel(NormBwdArgs a) {
  constexpr int E = Elem<T>::epc, NT = 1024;
  __shared__ float red[2][NT / 64];
  int par = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
    const T* dyr = static_cast<const T*>(a.dy) + t * a.d;
    const T* hr = static_cast<const T*>(a.h) + t * a.d;
    const float rs = a.rstd[t];
    float* p = a.part ? a.part + (int64_t)blockIdx.x * a.d : nullptr;
    float sum = 0.f;
    for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
      float y[E], n[E], w[E];
      unpack<T, E>(load_row_chunk(dyr, k, a.d), y);
      unpack<T, E>(load_row_chunk(hr, k, a.d), n);
      load_weight<E>(a.weight, k, a.d, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        n[e] *= rs;
        sum = fmaf(y[e] * w[e], n[e], sum);
        if (p && k + e < a.d) p[k + e] = t == (int64_t)blockIdx.x ? y[e] * n[e] : fmaf(y[e], n[e], p[k + e]);
      }
    }
    const float mean = row_sum<NT>(sum, red[par]) / (float)a.d;
    T* dxr = static_cast<T*>(a.dx) + t * a.d;
    for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
      float y[E], n[E], w[E], o[E];
      unpack<T, E>(load_row_chunk(dyr, k, a.d), y);
      unpack<T, E>(load_row_chunk(hr, k, a.d), n);
      load_weight<E>(a.weight, k, a.d, w);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = rs * fmaf(-(n[e] * rs), mean, y[e] * w[e]);
      if (a.dh) {
        float g[E];
        unpack<T, E>(load_row_chunk(static_cast<const T*>(a.dh) + t * a.d, k, a.d), g);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += g[e];
      }
      store_row_chunk<T>(dxr, k, a.d, o);
    }
  }
}

// (A launch holds less than 2^32 threads, which 2 d columns pass from d = 2^27 on:
// past kMostSums workgroups each takes several blocks of columns.)
constexpr unsigned kMostSums = 1u << 21;

__global__ __launch_bounds__(kSumThreads) void column_sum_kernel(ColumnSum s, unsigned groups) {
  for (unsigned b = blockIdx.x; b < groups; b += gridDim.x) {   // (uniform)
    column_sum(s, b);
    __syncthreads();
  }
}

template <typename T>
hipError_t launch_fwd(const NormArgs& a, hipStream_t st) {
  const RowShape r = forward_shape(a.T, a.d, Elem<T>::epc);
#define DORA_NORM(NT, C)                                                                                   \
  if (r.nt == NT && r.c == C) {                                                                            \
    const dim3 grid(grid_of(NT == 64 ? (a.T + 3) / 4 : a.T, NT)), block(NT == 64 ? 256 : NT);              \
    if (a.T * a.d * (int64_t)sizeof(T) <= kStreamBytes)                                                    \
      hipLaunchKernelGGL((rms_norm_kernel<T, NT, C, false, false>), grid, block, 0, st, a);                \
    else if (a.d * (int64_t)sizeof(T) % 128 != 0)                                                          \
      hipLaunchKernelGGL((rms_norm_kernel<T, NT, C, true, false>), grid, block, 0, st, a);                 \
    else                                                                                                   \
      hipLaunchKernelGGL((rms_norm_kernel<T, NT, C, true, true>), grid, block, 0, st, a);                  \
    return hipGetLastError();                                                                              \
  }
  DORA_NORM(64, 1)
  DORA_NORM(64, 2)
  DORA_NORM(256, 1)
  DORA_NORM(256, 2)
  DORA_NORM(512, 2)
  DORA_NORM(512, 4)
  DORA_NORM(1024, 1)
  DORA_NORM(1024, 2)
  if constexpr (Elem<T>::epc == 4) {
    DORA_NORM(1024, 4)
  }
#undef DORA_NORM
  hipLaunchKernelGGL((rms_norm_long_kernel<T>), dim3(grid_of(a.T, 1024)), dim3(1024), 0, st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_bwd(NormBwdArgs a, float* dweight, hipStream_t st) {
  const RowShape r = backward_shape(a.d, Elem<T>::epc);
  const int64_t grid = backward_grid(a.T, a.d, Elem<T>::epc);
  if (grid > 0) {
    hipError_t e = hipErrorInvalidValue;
    const bool stream = a.T * a.d * (int64_t)sizeof(T) > kStreamBytes && a.d * (int64_t)sizeof(T) % 128 == 0;
#define DORA_NORM_BWD(NT, C)                                                                            \
  if (r.nt == NT && r.c == C) {                                                                         \
    if (stream)                                                                                         \
      hipLaunchKernelGGL((rms_norm_bwd_kernel<T, NT, C, true>), dim3((unsigned)grid), dim3(NT), 0, st, a);  \
    else                                                                                                \
      hipLaunchKernelGGL((rms_norm_bwd_kernel<T, NT, C, false>), dim3((unsigned)grid), dim3(NT), 0, st, a); \
    e = hipGetLastError();                                                                              \
  }
    DORA_NORM_BWD(64, 1)
    DORA_NORM_BWD(256, 1)
    DORA_NORM_BWD(256, 2)
    DORA_NORM_BWD(512, 2)
    DORA_NORM_BWD(512, 4)
#undef DORA_NORM_BWD
    if (r.nt == 0) {
      hipLaunchKernelGGL((rms_norm_bwd_long_kernel<T>), dim3((unsigned)grid), dim3(1024), 0, st, a);
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  return dweight ? launch_column_sum(a.part, (int)grid, a.d, dweight, a.d, nullptr, st) : hipSuccess;
}

}  // namespace

hipError_t launch_column_sum(const float* part, int n_part, int64_t n, float* out0, int64_t n0, float* out1,
                             hipStream_t st) {
  const ColumnSum s{part, n_part, n, out0, n0, out1};
  const unsigned groups = sum_groups(n);
  hipLaunchKernelGGL(column_sum_kernel, dim3(groups < kMostSums ? groups : kMostSums), dim3(kSumThreads), 0, st, s,
                     groups);
  return hipGetLastError();
}

hipError_t launch_rms_norm(const void* x, const void* residual, const float* weight, float eps, int dtype, int64_t T,
                           int64_t d, void* h, void* y, void* q, float* scale, float* rstd, hipStream_t st) {
  const NormArgs a{x, residual, weight, eps, T, d, h, y, static_cast<uint8_t*>(q), scale, rstd};
  switch (dtype) {
    case 0: return launch_fwd<bf16_t>(a, st);
    case 2: return launch_fwd<f16_t>(a, st);
    default: return launch_fwd<float>(a, st);
  }
}

size_t rms_norm_bwd_workspace_bytes(int64_t T, int64_t d, int dtype) {
  return (size_t)(backward_grid(T, d, dtype == 1 ? 4 : 8) * d) * 4;
}

hipError_t launch_rms_norm_bwd(const void* dy, const void* dh, const void* h, const float* rstd, const float* weight,
                               int dtype, int64_t T, int64_t d, void* dx, float* dweight, void* ws, hipStream_t st) {
  const NormBwdArgs a{dy, dh, h, rstd, weight, T, d, dx, dweight ? static_cast<float*>(ws) : nullptr};
  switch (dtype) {
    case 0: return launch_bwd<bf16_t>(a, dweight, st);
    case 2: return launch_bwd<f16_t>(a, dweight, st);
    default: return launch_bwd<float>(a, dweight, st);
  }
}

}  // namespace dora
