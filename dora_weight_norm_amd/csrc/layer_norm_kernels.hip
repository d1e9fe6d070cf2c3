// The layer norm (layer_norm_device.h) and its backward on gfx950.
#include "layer_norm_device.h"

namespace dora {

namespace {

// ---------------------------------------------------------------------------
// Backward. With nh = (h - mean) rstd and a = dy w:
//   dx[t,j]    = rstd (a - mean_j(a) - nh mean_j(a nh)) + dh[t,j]
//   dweight[j] = sum_t dy nh           dbias[j] = sum_t dy
// dx is the gradient of x and of the residual alike. As the RMS norm's: a
// workgroup walks rows blockIdx.x, + gridDim.x, ... with its columns' weights
// and both sums in registers (rows in increasing order) and stores one partial
// row [dweight | dbias] at its end; a second kernel adds the partials in a
// fixed order. HBM bound: 8192 x 4096 bf16 with dh 53 us, 47 of them the rows
// (268 MB, 5.7 TB/s) and 4.5 the sums; twice or four times the workgroups, or
// stores past the caches, took 56 to 60.
// ---------------------------------------------------------------------------
struct LayerNormBwdArgs {
  const void* dy;
  const void* dh;
  const void* h;
  const float* mean;
  const float* rstd;
  const float* weight;
  int64_t T, d;
  void* dx;
  float* part;   // [gridDim.x][2][d], or null
};

// Both sums over the NT threads that share a row, in a fixed order.
template <int NT>
__device__ __forceinline__ void row_sum2(float& u, float& v, float* lds) {
  u = wave_sum(u), v = wave_sum(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) {
      lds[2 * (threadIdx.x >> 6)] = u;
      lds[2 * (threadIdx.x >> 6) + 1] = v;
    }
    __syncthreads();
    const int w = threadIdx.x & 15;
    u = row16_sum(w < NT / 64 ? lds[2 * w] : 0.f), v = row16_sum(w < NT / 64 ? lds[2 * w + 1] : 0.f);
  }
}

template <typename T, int NT, int C, bool STREAM>
__global__ __launch_bounds__(NT) void layer_norm_bwd_kernel(LayerNormBwdArgs a) {
  constexpr int E = Elem<T>::epc;
  __shared__ float red[2][NT > 64 ? 2 * (NT / 64) : 1];
  const int lane = threadIdx.x;
  constexpr bool KEEP = C <= 2;   // (no registers for the weights of four chunks)
  float w[KEEP ? C : 1][E], dw[C][E], db[C][E];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (KEEP) load_weight<E>(a.weight, (int64_t)(c * NT + lane) * E, a.d, w[c]);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[c][e] = db[c][e] = 0.f;
  }
  auto weight = [&](int c, float (&wc)[E]) __attribute__((always_inline)) {
    if constexpr (KEEP) {
#pragma unroll
      for (int e = 0; e < E; ++e) wc[e] = w[c][e];
    } else {
      load_weight<E>(reread(a.weight), (int64_t)(c * NT + lane) * E, a.d, wc);
    }
  };
  int par = 0;   // which words the row's sums go through: a wave a row ahead uses the other ones
  u32x4 yv[2][C], hv[2][C], gv[2][C];
  float mu2[2], rs2[2];
  // (a row's loads go out before the row ahead of it is reduced)
  auto load = [&](int64_t t, u32x4 (&y)[C], u32x4 (&h)[C], u32x4 (&g)[C], float& mu, float& rs)
      __attribute__((always_inline)) {
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
    mu = a.mean[t], rs = a.rstd[t];
  };
  auto row = [&](int64_t t, const u32x4 (&yr)[C], const u32x4 (&hr)[C], const u32x4 (&gr)[C], float mu, float rs)
      __attribute__((always_inline)) {
    float sa = 0.f, san = 0.f;   // (past d dy is 0, and with it every term)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float y[E], n[E];
      unpack<T, E>(yr[c], y);
      unpack<T, E>(hr[c], n);
      float wc[E];
      weight(c, wc);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        n[e] = (n[e] - mu) * rs;
        dw[c][e] = fmaf(y[e], n[e], dw[c][e]);
        db[c][e] += y[e];
        const float aw = y[e] * wc[e];
        sa += aw;
        san = fmaf(aw, n[e], san);
      }
    }
    row_sum2<NT>(sa, san, red[par]);
    par ^= 1;
    const float ma = sa / (float)a.d, man = san / (float)a.d;
    T* dxr = static_cast<T*>(a.dx) + t * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float y[E], n[E], o[E], wc[E];
      unpack<T, E>(yr[c], y);
      unpack<T, E>(hr[c], n);
      weight(c, wc);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = rs * fmaf(-((n[e] - mu) * rs), man, y[e] * wc[e] - ma);
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
  if constexpr (!KEEP) {   // (nor for a second row)
    for (; t < a.T; t += step) {
      load(t, yv[0], hv[0], gv[0], mu2[0], rs2[0]);
      row(t, yv[0], hv[0], gv[0], mu2[0], rs2[0]);
    }
  } else {
    if (t < a.T) load(t, yv[0], hv[0], gv[0], mu2[0], rs2[0]);
    for (; t < a.T; t += 2 * step) {
      if (t + step < a.T) load(t + step, yv[1], hv[1], gv[1], mu2[1], rs2[1]);
      row(t, yv[0], hv[0], gv[0], mu2[0], rs2[0]);
      if (t + step >= a.T) break;
      if (t + 2 * step < a.T) load(t + 2 * step, yv[0], hv[0], gv[0], mu2[0], rs2[0]);
      row(t + step, yv[1], hv[1], gv[1], mu2[1], rs2[1]);
    }
  }
  if (a.part) {
    float* p = a.part + (int64_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float v[4] = {dw[c][4 * i], dw[c][4 * i + 1], dw[c][4 * i + 2], dw[c][4 * i + 3]};
        const float u[4] = {db[c][4 * i], db[c][4 * i + 1], db[c][4 * i + 2], db[c][4 * i + 3]};
        store_row_chunk<float>(p, (int64_t)(c * NT + lane) * E + 4 * i, a.d, v);
        store_row_chunk<float>(p + a.d, (int64_t)(c * NT + lane) * E + 4 * i, a.d, u);
      }
  }
}

// Rows of any length: each row is read twice, and the workgroup's sums live in
// its partial row in memory (a thread adds to its own columns only, rows in
// increasing order).
template <typename T>
__global__ __launch_bounds__(1024) void layer_norm_bwd_long_kernel(LayerNormBwdArgs a) {
  constexpr int E = Elem<T>::epc, NT = 1024;
  __shared__ float red[2][2 * (NT / 64)];
  int par = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
    const T* dyr = static_cast<const T*>(a.dy) + t * a.d;
    const T* hr = static_cast<const T*>(a.h) + t * a.d;
    const float mu = a.mean[t], rs = a.rstd[t];
    float* p = a.part ? a.part + (int64_t)blockIdx.x * 2 * a.d : nullptr;
    const bool first = t == (int64_t)blockIdx.x;
    float sa = 0.f, san = 0.f;
    for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
      float y[E], n[E], w[E];
      unpack<T, E>(load_row_chunk(dyr, k, a.d), y);
      unpack<T, E>(load_row_chunk(hr, k, a.d), n);
      load_weight<E>(a.weight, k, a.d, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        n[e] = (n[e] - mu) * rs;
        const float aw = y[e] * w[e];
        sa += aw;
        san = fmaf(aw, n[e], san);
        if (p && k + e < a.d) {
          p[k + e] = first ? y[e] * n[e] : fmaf(y[e], n[e], p[k + e]);
          p[a.d + k + e] = first ? y[e] : p[a.d + k + e] + y[e];
        }
      }
    }
    row_sum2<NT>(sa, san, red[par]);
    const float ma = sa / (float)a.d, man = san / (float)a.d;
    T* dxr = static_cast<T*>(a.dx) + t * a.d;
    for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
      float y[E], n[E], w[E], o[E];
      unpack<T, E>(load_row_chunk(dyr, k, a.d), y);
      unpack<T, E>(load_row_chunk(hr, k, a.d), n);
      load_weight<E>(a.weight, k, a.d, w);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = rs * fmaf(-((n[e] - mu) * rs), man, y[e] * w[e] - ma);
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

template <typename T>
hipError_t launch_bwd(LayerNormBwdArgs a, float* dweight, float* dbias, hipStream_t st) {
  const RowShape r = backward_shape(a.d, Elem<T>::epc);
  const int64_t grid = backward_grid(a.T, a.d, Elem<T>::epc);
  if (grid > 0) {
    hipError_t e = hipErrorInvalidValue;
    const bool stream = a.T * a.d * (int64_t)sizeof(T) > kStreamBytes && a.d * (int64_t)sizeof(T) % 128 == 0;
#define DORA_NORM_BWD(NT, C)                                                                                  \
  if (r.nt == NT && r.c == C) {                                                                               \
    if (stream)                                                                                               \
      hipLaunchKernelGGL((layer_norm_bwd_kernel<T, NT, C, true>), dim3((unsigned)grid), dim3(NT), 0, st, a);  \
    else                                                                                                      \
      hipLaunchKernelGGL((layer_norm_bwd_kernel<T, NT, C, false>), dim3((unsigned)grid), dim3(NT), 0, st, a); \
    e = hipGetLastError();                                                                                    \
  }
    DORA_NORM_BWD(64, 1)
    DORA_NORM_BWD(256, 1)
    DORA_NORM_BWD(256, 2)
    DORA_NORM_BWD(512, 2)
    DORA_NORM_BWD(512, 4)
#undef DORA_NORM_BWD
    if (r.nt == 0) {
      hipLaunchKernelGGL((layer_norm_bwd_long_kernel<T>), dim3((unsigned)grid), dim3(1024), 0, st, a);
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  return dweight || dbias ? launch_column_sum(a.part, (int)grid, 2 * a.d, dweight, a.d, dbias, st) : hipSuccess;
}

}  // namespace

hipError_t launch_layer_norm(const void* x, const void* residual, const float* weight, const float* bias, float eps,
                             int dtype, int64_t T, int64_t d, void* h, void* y, void* q, int q_int8, float* scale,
                             float* mean, float* rstd, hipStream_t st) {
  const LayerNormArgs a{x, residual, weight, bias, eps, T, d, h, y, q, q_int8 ? kQInt8 : kQE4m3, scale, mean, rstd};
  return launch_rows<true>(a, dtype, st);
}

size_t layer_norm_bwd_workspace_bytes(int64_t T, int64_t d, int dtype) {
  return (size_t)(backward_grid(T, d, dtype == 1 ? 4 : 8) * 2 * d) * 4;
}

hipError_t launch_layer_norm_bwd(const void* dy, const void* dh, const void* h, const float* mean, const float* rstd,
                                 const float* weight, int dtype, int64_t T, int64_t d, void* dx, float* dweight,
                                 float* dbias, void* ws, hipStream_t st) {
  const LayerNormBwdArgs a{dy, dh, h, mean, rstd, weight, T, d, dx,
                           dweight || dbias ? static_cast<float*>(ws) : nullptr};
  switch (dtype) {
    case 0: return launch_bwd<bf16_t>(a, dweight, dbias, st);
    case 2: return launch_bwd<f16_t>(a, dweight, dbias, st);
    default: return launch_bwd<float>(a, dweight, dbias, st);
  }
}

}  // namespace dora
